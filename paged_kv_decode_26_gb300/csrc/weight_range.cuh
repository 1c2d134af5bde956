// weight_range.cuh -- the numbers that softmax weights are kept as on their way
// into the second product.
//
// A weight is 2^((x - m) + LIFT) with m a running reference: the largest score
// at the time it was set, and set again once a score lies more than GROW above
// it.  (So the common tile or chunk needs no rescaling of O.)  Weights then
// reach 2^(LIFT + GROW), and the sum and O carry the same factor, which cancels
// in O / l; states (m, l) that leave a kernel carry l / 2^LIFT.
// m itself is a score, never shifted: where fp32 no longer resolves LIFT or
// GROW beside it (from 2^24 on), x - m is still exact, and 0 for the key that
// set m.
//   bf16  has fp32's exponents, and values up to the end of fp32's range, which
//         their weighted sum O leaves before it is divided by l.  Lowered by
//         2^17 O stays within it up to l = 2^17 of the largest weight; weights
//         then vanish below 2^-109, and results below 2^-109.  (17 and not 16:
//         around -17 fp32's steps are as coarse as those of LIFT - m for m in
//         -49 .. 15, so m + (LIFT - m) rounds to LIFT and a lone key's weight
//         divides out to the last bit of an fp32 output.)
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
    static constexpr float LIFT = -17.f, GROW = 8.f;
    static constexpr float UNLIFT = 131072.f;             // 2^-LIFT
};
template <>
struct WeightRange<__half> {
    static constexpr float LIFT = 11.f, GROW = 4.f;
    static constexpr float UNLIFT = 1.f / 2048.f;
};

// The reference of one row of the softmax on tcgen05.  With y the raw products
// and x = a y the scores (a > 0), the exponent of a weight is one multiply-add,
// a y + add, as long as its roundings are far below 1 (2^-9 up to |m| = 2^15,
// less than those of the products beside them).  The unrounded a y of the key
// that set m may exceed m by half m's last bit, a factor of 2^8 in a weight at
// 2^27: an item with a reference beyond() goes on with y replaced by x, rounded,
// and a by 1.  Beyond 2^23, where fp32 holds no fractions and soon not LIFT - m,
// there is no lift and nothing to grow by (weights stay at 1 or below).
template <typename T>
struct RowReference {
    using Range = WeightRange<T>;
    float m = -INFINITY;
    float add = 0.f;
    float grow = Range::GROW;

    // (-inf - -inf is NaN: no key seen yet, or nothing to see)
    __device__ __forceinline__ bool exceeded(float x) const { return x - m > grow; }
    __device__ __forceinline__ static bool beyond(float x) { return fabsf(x) > 32768.f; }
    __device__ __forceinline__ static float lift(float m) {
        return fabsf(m) <= 8388608.f ? Range::LIFT : 0.f;
    }
    // What the sum is to be multiplied by beside m.
    __device__ __forceinline__ static float unit(float m) {
        return fabsf(m) <= 8388608.f ? Range::UNLIFT : 1.f;
    }
    // Takes in the largest score of a tile; the factor for what the row has
    // summed up so far.
    __device__ __forceinline__ float take(float x) {
        if (!exceeded(x)) return 1.f;
        const float alpha = m == -INFINITY ? 1.f : exp2f((m - x) + (lift(x) - lift(m)));
        m = x;
        add = lift(x) - x;
        grow = fabsf(x) <= 8388608.f ? Range::GROW : 0.f;
        return alpha;
    }
};

}  // namespace pkv
