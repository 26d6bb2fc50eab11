#define HEAD_DIM 64
#include "chunk_dim.inc"
