// decode_shared_f16.cu -- shared-prefix decode kernels for f16.
#define PKV_ELEM __half
#define PKV_FN launch_shared_f16
#include "decode_shared_inst.inc"
