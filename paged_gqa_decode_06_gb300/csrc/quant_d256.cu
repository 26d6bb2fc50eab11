#define HEAD_DIM 256
#include "quant_dim.inc"
