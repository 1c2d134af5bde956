// decode_pieces_bf16.cu -- piece decode kernels for bf16 queries and K/V.
#define PKV_ELEM __nv_bfloat16
#define PKV_FN launch_pieces_bf16
#include "decode_pieces_inst.inc"
