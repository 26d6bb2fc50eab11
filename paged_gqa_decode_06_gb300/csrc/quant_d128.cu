#define HEAD_DIM 128
#include "quant_dim.inc"
