// decode_q8_launch.h -- host-side launch interface of decode_q8_kernel, one
// translation unit per type of the queries.
#pragma once

#include "decode_q8_kernel.cuh"

namespace pkv {

struct Q8Launch {
    CUtensorMap tm_k;     // boxes of 16 tokens of one kv head
    CUtensorMap tm_v;
    Q8Params p;
    int whole;            // warps per context of decode_q8_short_kernel; 0: decode_q8_kernel
    cudaStream_t stream;
};

// Launch decode_q8_kernel<D, T> or decode_q8_short_kernel<D, T>.
cudaError_t launch_decode_q8_bf16(int D, const Q8Launch& L);
cudaError_t launch_decode_q8_f16(int D, const Q8Launch& L);

}  // namespace pkv
