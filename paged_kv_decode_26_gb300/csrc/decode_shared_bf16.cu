// decode_shared_bf16.cu -- shared-prefix decode kernels for bf16.
#define PKV_ELEM __nv_bfloat16
#define PKV_FN launch_shared_bf16
#include "decode_shared_inst.inc"
