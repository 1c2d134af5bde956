// attn_prompt_bf16.cu -- tcgen05 attention kernels of whole prompts for bf16.
#define PKV_ELEM __nv_bfloat16
#define PKV_FN launch_attn_prompt_bf16
#include "attn_prompt_inst.inc"
