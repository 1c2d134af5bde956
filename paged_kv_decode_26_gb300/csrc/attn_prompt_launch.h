// attn_prompt_launch.h -- host-side launch interface of attn_prompt_kernel
// (attn_prompt_kernel.cuh).
#pragma once

#include "attn_prompt_kernel.cuh"

namespace pkv {

struct AttnLaunch {
    CUtensorMap tm_q;
    CUtensorMap tm_k;
    CUtensorMap tm_v;
    CUtensorMap tm_o;
    AttnParams p;
    int ctas;
    size_t smem_bytes;
    cudaStream_t stream;
};

// Launch attn_prompt_kernel<D, T, precise>.
cudaError_t launch_attn_prompt_bf16(int D, bool precise, const AttnLaunch& L);
cudaError_t launch_attn_prompt_f16(int D, bool precise, const AttnLaunch& L);

}  // namespace pkv
