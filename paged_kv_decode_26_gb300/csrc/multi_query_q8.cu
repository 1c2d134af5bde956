// multi_query_q8.cu -- instances of the multi-query kernel over 8-bit pages.
#include "decode_launch.h"
#include "multi_query_q8_launch.h"

namespace pkv {
namespace {

template <int D, int BS, int PARTS>
cudaError_t launch(const Mq8Launch& L) {
    static unsigned long long done_mask = 0;
    static bool split_fits = false;
    const void* fn = reinterpret_cast<const void*>(&multi_query_q8_kernel<D, BS, PARTS>);
    const size_t smem = Mq8Sizes<D>::SMEM;
    cudaError_t e;
    if (!split_fits) {
        // the warps' shares of the registers add up to those of the launch, or the
        // kernel would wait for registers for ever
        cudaFuncAttributes a;
        if ((e = cudaFuncGetAttributes(&a, fn)) != cudaSuccess) return e;
        if (a.numRegs * kMq8Threads < 256 * (kMq8SoftmaxRegs + kMq8OtherRegs))
            return cudaErrorInvalidConfiguration;
        split_fits = true;
    }
    if ((e = ensure_smem_limit(fn, &done_mask, smem)) != cudaSuccess) return e;
    multi_query_q8_kernel<D, BS, PARTS><<<L.ctas, kMq8Threads, smem, L.stream>>>(L.p);
    return cudaGetLastError();
}

template <int PARTS>
cudaError_t by_shape(int D, int BS, const Mq8Launch& L) {
    if (D == 64) return BS == 16 ? launch<64, 16, PARTS>(L) : launch<64, 32, PARTS>(L);
    return BS == 16 ? launch<128, 16, PARTS>(L) : launch<128, 32, PARTS>(L);
}

}  // namespace

cudaError_t launch_multi_query_q8(int D, int BS, const Mq8Launch& L) {
    return L.p.out_dtype == PKV_F32 ? by_shape<2>(D, BS, L) : by_shape<1>(D, BS, L);
}

}  // namespace pkv
