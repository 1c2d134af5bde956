// decode_weights_launch.h -- host-side launch interface of
// decode_pieces_kernel with weights, one translation unit per
// element type.
#pragma once

#include "decode_pieces_kernel.cuh"

namespace pkv {

struct PiecesLaunch {
    CUtensorMap tm_k;     // chunks of one kv head
    CUtensorMap tm_v;
    PieceParams p;
    cudaStream_t stream;
};

// Launch decode_pieces_kernel<D, T, true>.
cudaError_t launch_weights_bf16(int D, const PiecesLaunch& L);
cudaError_t launch_weights_f16(int D, const PiecesLaunch& L);

}  // namespace pkv
