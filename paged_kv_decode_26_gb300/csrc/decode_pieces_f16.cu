// decode_pieces_f16.cu -- piece decode kernels for f16 queries and K/V.
#define PKV_ELEM __half
#define PKV_FN launch_pieces_f16
#include "decode_pieces_inst.inc"
