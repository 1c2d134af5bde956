// decode_pieces_launch.h -- host-side launch interface of the piece decode
// (decode_pieces_kernel.cuh), one translation unit per element type.
#pragma once

#include "decode_pieces_kernel.cuh"

namespace pkv {

struct PiecesLaunch {
    CUtensorMap tm_k;     // boxes of [16 tokens x 64 elements] of one kv head
    CUtensorMap tm_v;
    PieceParams p;
    int ctas;
    bool after_prefix;    // overlaps the prefix kernel ahead of it on the stream
    cudaStream_t stream;
};

// Launch decode_pieces_kernel<D, T, weights>.
cudaError_t launch_pieces_bf16(int D, bool weights, const PiecesLaunch& L);
cudaError_t launch_pieces_f16(int D, bool weights, const PiecesLaunch& L);

}  // namespace pkv
