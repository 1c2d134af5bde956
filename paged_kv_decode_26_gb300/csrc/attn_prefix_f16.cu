// attn_prefix_f16.cu -- tcgen05 attention kernels of shared prefixes for f16.
#define PKV_ELEM __half
#define PKV_PAGED true
#define PKV_FN launch_attn_prefix_f16
#include "attn_tc_inst.inc"
