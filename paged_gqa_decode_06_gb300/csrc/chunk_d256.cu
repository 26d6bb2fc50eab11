#define HEAD_DIM 256
#include "chunk_dim.inc"
