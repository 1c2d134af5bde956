// weight_range.cuh -- the numbers that softmax weights are kept as on their way
// into the second product.
//
// A weight is 2^(x - m) with m a running reference: LIFT below the largest score
// at the time it was set, and set again once a score lies more than GROW above
// that one.  (So the common tile or chunk needs no rescaling of O.)  Weights
// then reach 2^(LIFT + GROW), and the sum and O carry the same factor, which
// cancels in O / l and in merges of (m, l) states.
//   bf16  has fp32's exponents: no lift.
//   fp16  is spaced by 2^-24 at best.  Without a lift weights below 2^-14 lose
//         bits one by one and those below 2^-25 vanish -- thousands of keys of
//         small weight beside one of large weight would not add up (1500 keys
//         at 2^-10 .. 2^-19: off by up to 2^-6 of their sum).  Lifted by 2^11 and
//         let grow by 2^4, below fp16's largest 2^16, the spacing is 2^-35 of the
//         largest weight.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

template <typename T>
struct WeightRange;
template <>
struct WeightRange<__nv_bfloat16> {
    static constexpr float LIFT = 0.f, GROW = 8.f;
};
template <>
struct WeightRange<__half> {
    static constexpr float LIFT = 11.f, GROW = 4.f;
};

}  // namespace pkv
