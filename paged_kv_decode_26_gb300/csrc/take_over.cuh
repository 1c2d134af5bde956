// take_over.cuh -- a running CTA takes over the work of CTAs of its grid that
// have not started (cluster launch control, sm_100 and later): dynamic work
// distribution without a counter in memory, so a launch needs no workspace
// for it and launches that overlap do not meet.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// Asks for a CTA of this grid that has not started; the answer (16 bytes)
// completes on `bar`.  If there was one it will not start: the caller does its
// work.  No request may follow one that found none.
__device__ __forceinline__ void steal_cta(uint4* answer, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
        "[%0], [%1];" ::"r"(smem_addr(answer)),
        "r"(smem_addr(bar))
        : "memory");
}
// Index of the CTA taken over, -1 if there was none left.
__device__ __forceinline__ int stolen_cta(const uint4* answer) {
    int id;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 x;\n\t"
        "ld.shared.b128 h, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "mov.b32 x, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 x, h;\n\t"
        "mov.b32 %0, x;\n\t}"
        : "=r"(id)
        : "r"(smem_addr(answer))
        : "memory");
    // the next answer is written by the async proxy after this read
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    return id;
}

}  // namespace pkv
