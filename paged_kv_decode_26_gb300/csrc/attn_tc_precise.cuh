// attn_tc_precise.cuh -- the products and the softmax of attn_tc_kernel.cuh for
// fp32 outputs.  They need more in two places:
//
//   weights   a softmax weight enters the second product as the sum of as many
//             16-bit parts as fp32 needs: two of fp16 (22 bits), three of bf16
//             (24), each the rounding of what the ones before leave.
//   sums      the tensor core drops the bits of a product below its
//             accumulator's last one, always downwards: over 32768 keys O came
//             out 2e-4 short.  So O of each key tile starts from zero, smallest
//             parts first, and joins a sum in registers by fp32 additions (7e-7
//             at 32768 keys).
//
// Tensor memory then has room for one row tile: O of a key tile (D columns) and
// two buffers of S and P (192 columns each: S or two parts, and the third), so
// that S of the next key tile is there when the softmax is done with this one.
// Warps 0-3 are the softmax, a thread per row; warps 4-7 hold the sums, a thread
// per row, and write the output.  What bounds it: the softmax, 4000 cycles a key
// tile of which 3000 (bf16; fp16 2260) form and store P's parts, one warp per
// scheduler; the tensor core's 3 or 4 products of 128 x 128 x D take 1536 or
// 2048.  GB300, sixteen prompts of 128-2048 tokens, 32/8 heads of 128: 480 us
// (fp16 418); with O summed in tensor memory by the softmax warps, in turn with
// everything else, 672 (507).
#pragma once

#include "attn_tc_kernel.cuh"

namespace pkv {

constexpr int kAtAlphas = 4;      // key tiles whose rescaling factors are kept

template <typename T>
__host__ __device__ constexpr int attn_parts() {
    return std::is_same<T, __nv_bfloat16>::value ? 3 : 2;
}
// Columns of S and P (part k at 64 k) for key tile g of the CTA.
__device__ __forceinline__ uint32_t attn_buffer_col(uint32_t g) { return 128u + (g & 1u) * 192u; }

// Between the softmax and the sums, behind the output rows of warps 4-7:
// alpha[g % 4][row], 2^(reference before key tile g - reference after);
// (reference, sum of weights)[item slot][row].
__device__ __forceinline__ float* attn_alphas(const AttnControl& ctl) {
    return reinterpret_cast<float*>(ctl.sOut + 4 * 32 * 128);
}
__device__ __forceinline__ float2* attn_rows(const AttnControl& ctl) {
    return reinterpret_cast<float2*>(attn_alphas(ctl) + kAtAlphas * kAtRows);
}

// Warp 8: every MMA.  The CTA's key tiles are numbered through its items; S
// runs one tile ahead of P V.
template <int D, typename T, bool PAGED>
__device__ __forceinline__ void attn_mma_precise(const AttnControl& ctl, const AttnParams& p,
                                                 int lane) {
    PKV_ATTN_SIZES(D)
    constexpr int PARTS = attn_parts<T>();
    const uint32_t id_s = tc_idesc<T>(kAtRows, kAtKeys, 0);
    const uint32_t id_o = tc_idesc<T>(kAtRows, D, 1);
    const uint64_t dq0 = tc_desc_sw128(smem_addr(ctl.sQ), 16, 1024);
    const uint64_t dk0 = tc_desc_sw128(smem_addr(ctl.sKV), 16, 1024);
    const uint64_t dv0 = tc_desc_sw128(smem_addr(ctl.sKV), KV_HALF, 1024);
    const uint32_t lead = elect_one() ? 1u : 0u;
    int slot = 0, sph = 0;              // item ring
    int kst = 0, vst = 1;               // ring slots of the next K and V tile
    uint32_t kph = 0, vph = 0;
    int nt = 0, j = 0;                  // key tiles of S's item, and the next one
    uint32_t n_items = 0, n_s = 0;      // items and key tiles whose S is issued
    bool ok = true, more = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, p.errors));
    };
    auto advance2 = [&](int& st, uint32_t& ph) {
        st += 2;
        if (st >= ctl.stages) {
            st -= ctl.stages;
            ph ^= 1u;
        }
    };
    // the next item with products
    auto next_item = [&]() {
        for (;;) {
            wait(&ctl.it_full[slot], sph);
            if (!ok) return;
            const bool done = ctl.items[slot].done != 0;
            const bool skip = PAGED && ctl.items[slot].split < 0;
            nt = ctl.items[slot].nt[0];
            __syncwarp();
            if (done) {
                more = false;
                return;
            }
            if (lane == 0) mbar_arrive(&ctl.it_free[slot]);
            if (++slot == kAtItems) {
                slot = 0;
                sph ^= 1;
            }
            if (!skip) return;
        }
    };
    auto issue_s = [&]() {
        if (!more) return;
        if (j == nt) {
            if (n_s > 0) ++n_items;
            next_item();
            if (!ok || !more) return;
            j = 0;
            wait(&ctl.q_full[n_items & 1], n_items >> 1);
        }
        wait(&ctl.kv_full[kst], kph);
        if (!ok) return;
        tc_fence_after();
        const uint64_t q = dq0 + (uint64_t)((n_items & 1) * (Q_BYTES >> 4));
        const uint64_t k = dk0 + (uint64_t)(kst * (KV_BYTES >> 4));
        const uint32_t d = ctl.tmem + attn_buffer_col(n_s);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            at_mma(d, q + (((i / 4) * Q_HALF + (i % 4) * 32) >> 4),
                   k + (((i / 4) * KV_HALF + (i % 4) * 32) >> 4), id_s, i > 0 ? 1u : 0u, lead);
        at_commit(&ctl.s_full[n_s & 1], lead);
        at_commit(&ctl.kv_free[kst], lead);
        if (j + 1 == nt) at_commit(&ctl.q_free[n_items & 1], lead);
        __syncwarp();
        advance2(kst, kph);
        ++j;
        ++n_s;
    };
    issue_s();
    for (uint32_t g = 0; ok && g < n_s; ++g) {
        issue_s();
        if (g > 0) wait(&ctl.o_free[0], g - 1);
        wait(&ctl.kv_full[vst], vph);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            wait(&ctl.p_full[2 * (g & 1) + half], g >> 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = ctl.tmem + attn_buffer_col(g);
            const uint64_t v = dv0 + (uint64_t)(vst * (KV_BYTES >> 4));
#pragma unroll
            for (int part = PARTS - 1; part >= 0; --part)
#pragma unroll
                for (int i = half * 4; i < half * 4 + 4; ++i)
                    at_mma_tmem_a(ctl.tmem, a + part * 64 + i * 8,
                                  v + (uint64_t)((i * 16 * 128) >> 4), id_o,
                                  (part < PARTS - 1 || i > 0) ? 1u : 0u, lead);
            __syncwarp();
        }
        if (!ok) break;
        at_commit(&ctl.o_full[0], lead);
        at_commit(&ctl.kv_free[vst], lead);
        __syncwarp();
        advance2(vst, vph);
    }
    // every MMA complete before the tensor memory is released
    at_commit(ctl.fin, lead);
    __syncwarp();
    mbar_wait(ctl.fin, 0, p.errors);
    __syncwarp();
}

// Warps 0-3: thread r owns row r.
template <int D, typename T, bool PAGED>
__device__ __forceinline__ void attn_softmax_precise(const AttnControl& ctl, const AttnParams& p,
                                                     int warp, int lane) {
    PKV_ATTN_SIZES(D)
    constexpr int PARTS = attn_parts<T>();
    const int G = p.group;
    const int r = warp * 32 + lane;
    const uint32_t t_lane = ctl.tmem + ((uint32_t)(warp * 32) << 16);
    const float sc = p.scale_log2;
    int slot = 0, sph = 0;
    uint32_t g = 0;                                   // key tiles of the CTA so far
    bool ok = true;
    while (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.it_full[slot], sph, p.errors));
        if (!ok) break;
        const AttnItem it = ctl.items[slot];
        if (it.done) break;
        const int nt = PAGED && it.split < 0 ? 0 : it.nt[0];
        // last key this row sees
        const int pos = PAGED ? it.n_keys - 1 : it.pos0 + r / G;
        const int warp_pos = PAGED ? pos : it.pos0 + (warp * 32) / G;
        RowReference<T> ref;
        float2 l4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) l4[i] = make_float2(0.f, 0.f);
        for (int j = 0; j < nt; ++j, ++g) {
            ok = __all_sync(0xffffffffu, mbar_wait(&ctl.s_full[g & 1], (g >> 1) & 1u, p.errors));
            if (!ok) break;
            tc_fence_after();
            const uint32_t buf = t_lane + attn_buffer_col(g);
            float y[kAtKeys];
            uint32_t* yr = reinterpret_cast<uint32_t*>(y);
            tc_ld32(buf, yr);
            tc_ld32(buf + 32, yr + 32);
            tc_ld32(buf + 64, yr + 64);
            tc_ld32(buf + 96, yr + 96);
            tc_wait_ld();
            // scores, rounded (the exponent from the product in one multiply-add
            // fails for large ones, see RowReference; prompts take the same time)
            const float2 sc2 = make_float2(sc, sc);
#pragma unroll
            for (int c = 0; c < kAtKeys; c += 2) {
                const float2 x = __fmul2_rn(make_float2(y[c], y[c + 1]), sc2);
                y[c] = x.x;
                y[c + 1] = x.y;
            }
            if (j * kAtKeys + kAtKeys - 1 > warp_pos) {
                // keys that rows of this warp may not see
                const int lim = pos - j * kAtKeys;
#pragma unroll
                for (int c = 0; c < kAtKeys; ++c) y[c] = c <= lim ? y[c] : -INFINITY;
            }
            float m8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) m8[e] = fmaxf(y[e], y[8 + e]);
#pragma unroll
            for (int c = 16; c < kAtKeys; c += 16)
#pragma unroll
                for (int e = 0; e < 8; ++e) m8[e] = max3(m8[e], y[c + e], y[c + 8 + e]);
            const float mx = max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]),
                                  fmaxf(m8[6], m8[7]));
            float alpha = 1.f;
            if (ref.exceeded(mx)) {
                alpha = ref.take(mx);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    l4[i] = __fmul2_rn(l4[i], make_float2(alpha, alpha));
            }
            attn_alphas(ctl)[(g % kAtAlphas) * kAtRows + r] = alpha;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.alpha_full[g % kAtAlphas]);
            const float2 add = make_float2(ref.add, ref.add);
            const float2 neg1 = make_float2(-1.f, -1.f);
#pragma unroll
            for (int quarter = 0; quarter < 4; ++quarter) {
                uint32_t w[PARTS][16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int c = 2 * (quarter * 16 + i);
                    const float2 e = __fadd2_rn(make_float2(y[c], y[c + 1]), add);
                    float2 pv = make_float2(exp2f(e.x), exp2f(e.y));
                    l4[i & 3] = __fadd2_rn(l4[i & 3], pv);
#pragma unroll
                    for (int k = 0; k < PARTS; ++k) {
                        w[k][i] = pack2<T>(pv.x, pv.y);
                        if (k + 1 < PARTS) pv = __ffma2_rn(unpack2<T>(w[k][i]), neg1, pv);
                    }
                }
#pragma unroll
                for (int k = 0; k < PARTS; ++k) tc_st16(buf + k * 64 + quarter * 16, w[k]);
                if (quarter & 1) {
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.p_full[2 * (g & 1) + quarter / 2]);
                }
            }
        }
        if (!ok) break;
        const float2 la = __fadd2_rn(l4[0], l4[1]), lb = __fadd2_rn(l4[2], l4[3]);
        attn_rows(ctl)[slot * kAtRows + r] = make_float2(ref.m, (la.x + lb.x) + (la.y + lb.y));
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&ctl.row_full[slot]);
            mbar_arrive(&ctl.it_free[slot]);
        }
        if (++slot == kAtItems) {
            slot = 0;
            sph ^= 1;
        }
    }
    __syncwarp();
}

// Warps 4-7: thread r sums row r of O over the key tiles and writes it.
template <int D, typename T, bool PAGED>
__device__ __forceinline__ void attn_sum_precise(const AttnControl& ctl, const AttnParams& p,
                                                 const CUtensorMap& tm_o, int warp, int lane) {
    PKV_ATTN_SIZES(D)
    const int G = p.group;
    const int warp_row = (warp - 4) * 32, r = warp_row + lane;
    const uint32_t t_lane = ctl.tmem + ((uint32_t)warp_row << 16);
    unsigned char* stage = ctl.sOut + (warp - 4) * 32 * 128;
    int slot = 0, sph = 0;
    uint32_t g = 0;
    bool ok = true;
    while (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.it_full[slot], sph, p.errors));
        if (!ok) break;
        const AttnItem it = ctl.items[slot];
        if (it.done) break;
        const bool bad = PAGED && it.split < 0;
        const int nt = bad ? 0 : it.nt[0];
        float sum[D];
#pragma unroll
        for (int c = 0; c < D; ++c) sum[c] = 0.f;
        for (int j = 0; j < nt; ++j, ++g) {
            bool w = mbar_wait(&ctl.alpha_full[g % kAtAlphas], (g / kAtAlphas) & 1u, p.errors);
            w = w && mbar_wait(&ctl.o_full[0], g & 1u, p.errors);
            ok = __all_sync(0xffffffffu, w);
            if (!ok) break;
            tc_fence_after();
            const float alpha = attn_alphas(ctl)[(g % kAtAlphas) * kAtRows + r];
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                tc_ld32(t_lane + c0, o);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    sum[c0 + c] = fmaf(sum[c0 + c], alpha, __uint_as_float(o[c]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.o_free[0]);
        }
        if (!ok) break;
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.row_full[slot], sph, p.errors));
        if (!ok) break;
        const float2 ml = attn_rows(ctl)[slot * kAtRows + r];
        const float inv = ml.y != 0.f ? 1.f / ml.y : 0.f;
        const int tok = r / G;                         // within the item
        const bool real = tok < it.rows;
        const bool all = (warp_row + 31) / G < it.rows;
        const int split = bad ? -1 - it.split : it.split;
        const size_t row = (size_t)(it.row0 + tok) * p.n_heads + it.kvh * G + r % G;
        const size_t unit = PAGED ? row * p.max_splits + split : row;
        if (PAGED && real)
            *reinterpret_cast<float2*>(p.pre_ml + unit * 2) =
                make_float2(ml.x, ml.y * RowReference<T>::unit(ml.x));
        const bool poison = !PAGED && ctl.poison[slot] != 0;
        unsigned char* own = static_cast<unsigned char*>(PAGED ? p.pre_o : p.out) + unit * D * 4;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
            uint32_t w[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) w[c] = __float_as_uint(sum[q * 32 + c] * inv);
            if (poison) {
                // NaN and infinities that the guard took out of V, from the
                // rows that this query sees
#pragma unroll 1
                for (int key = it.pos0 / kAtKeys * kAtKeys;
                     key <= min(it.pos0 + tok, it.n_keys - 1); ++key) {
                    const T* v = static_cast<const T*>(p.v) +
                                 (size_t)(it.key_row + key) * p.v_stride + it.kvh * D + q * 32;
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float x = to_float<T>(v[c]);
                        if (!at_finite(x)) w[c] = __float_as_uint(__uint_as_float(w[c]) + x);
                    }
                }
            }
            attn_store(tm_o, stage, own + q * 128, w, all, real,
                       q + (PAGED ? split * (D / 32) : 0), it.kvh * G, it.row0 + warp_row / G,
                       lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.it_free[slot]);
        if (++slot == kAtItems) {
            slot = 0;
            sph ^= 1;
        }
    }
    if (lane == 0) bulk_wait();
    __syncwarp();
}

}  // namespace pkv
