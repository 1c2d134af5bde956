// decode_q8_bf16.cu -- 8-bit decode kernels for bf16 queries.
#define PKV_ELEM __nv_bfloat16
#define PKV_FN launch_decode_q8_bf16
#include "decode_q8_inst.inc"
