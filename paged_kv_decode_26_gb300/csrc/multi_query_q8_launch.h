// multi_query_q8_launch.h -- host-side launch interface of multi_query_q8_kernel.
#pragma once

#include "multi_query_q8_kernel.cuh"

namespace pkv {

struct Mq8Launch {
    Mq8Params p;
    unsigned ctas;
    cudaStream_t stream;
};

// Launch multi_query_q8_kernel<D, BS>.
cudaError_t launch_multi_query_q8(int D, int BS, const Mq8Launch& L);

}  // namespace pkv
