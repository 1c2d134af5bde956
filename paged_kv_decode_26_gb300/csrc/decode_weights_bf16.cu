// decode_weights_bf16.cu -- weight-accumulating decode kernels for bf16.
#define PKV_ELEM __nv_bfloat16
#define PKV_FN launch_weights_bf16
#include "decode_weights_inst.inc"
