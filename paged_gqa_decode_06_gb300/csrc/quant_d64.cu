#define HEAD_DIM 64
#include "quant_dim.inc"
