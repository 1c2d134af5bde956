// decode_shared_launch.h -- host-side launch interface of the shared-prefix
// decode (decode_shared_kernel.cuh, decode_pieces_kernel.cuh).
#pragma once

#include "decode_pieces_kernel.cuh"
#include "decode_shared_kernel.cuh"

namespace pkv {

struct SharedLaunch {
    CUtensorMap tm_q;
    CUtensorMap tm_k;      // whole pages of one kv head
    CUtensorMap tm_v;
    CUtensorMap tm_o;      // the prefixes' partial outputs
    CUtensorMap tm_kc;     // chunks of one kv head
    CUtensorMap tm_vc;
    AttnParams a;
    PieceParams p;
    int prefix_ctas;       // 0: no prefixes
    cudaStream_t stream;
};

// Launch decode_pieces_kernel<D, T, false, false, precise> and, as SMs get free of it,
// attn_prefix_kernel<D, T, precise>.
cudaError_t launch_shared_bf16(int D, bool precise, const SharedLaunch& L);
cudaError_t launch_shared_f16(int D, bool precise, const SharedLaunch& L);

}  // namespace pkv
