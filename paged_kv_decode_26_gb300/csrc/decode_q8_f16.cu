// decode_q8_f16.cu -- 8-bit decode kernels for fp16 queries.
#define PKV_ELEM __half
#define PKV_FN launch_decode_q8_f16
#include "decode_q8_inst.inc"
