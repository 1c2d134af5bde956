// attn_prefix_bf16.cu -- tcgen05 attention kernels of shared prefixes for bf16.
#define PKV_ELEM __nv_bfloat16
#define PKV_PAGED true
#define PKV_FN launch_attn_prefix_bf16
#include "attn_tc_inst.inc"
