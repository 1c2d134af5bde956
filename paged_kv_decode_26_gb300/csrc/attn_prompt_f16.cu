// attn_prompt_f16.cu -- tcgen05 attention kernels of whole prompts for f16.
#define PKV_ELEM __half
#define PKV_FN launch_attn_prompt_f16
#include "attn_prompt_inst.inc"
