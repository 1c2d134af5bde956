// decode_weights_f16.cu -- weight-accumulating decode kernels for f16.
#define PKV_ELEM __half
#define PKV_FN launch_weights_f16
#include "decode_weights_inst.inc"
