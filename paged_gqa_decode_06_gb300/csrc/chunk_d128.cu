#define HEAD_DIM 128
#include "chunk_dim.inc"
