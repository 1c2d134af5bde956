// decode_q8_kernel.cuh -- paged decode over 8-bit pages (e4m3 with a scale per
// block and kv head) as equal pieces per warp (sm_103a): paged_attn_decode_q8.
//
// Mathematics: with codes k_t, v_t and the scales a_t, b_t of token t's block,
// scores x_t = scale log2(e) a_t (q . k_t), the sum L of p_t = 2^(x_t - m) and
// O = sum p_t b_t v_t; the result is O / L.  Codes are exact in fp16, so they
// enter mma.sync as they are and the scales stay in fp32: a_t on the score, b_t on
// the weight.
//
// What bounds it: HBM, at half the bytes of 16-bit pages for the same products, so
// twice the work a byte.  A 32-token chunk of one kv head (8 KB) is 16 + 32
// products m16n8k16, 128 conversions of two codes and 16 ldmatrix.  Measured: 16
// contexts of 8K-32K, 32 heads of 128, 414-434 us (6.6-6.9 TB/s), 128 of 16-8192, 32 query
// and 8 kv heads, 171-179 us (6.2-6.5 TB/s); 4 of up to 200 tokens 5.0 us.  fp32 outputs
// take as long.
//
// Layout: the tokens are the rows of the score product and the inner dimension of
// the second one.  An ldmatrix of 16-bit units hands a lane bytes 4 t .. 4 t + 3
// of a token's 16 dims, which two conversions turn into two registers of the A
// operand; the inner dimension's order is the queries' to choose (MMA columns
// 2 t, 2 t + 1 stand for dims 4 t, 4 t + 1, columns 2 t + 8, + 9 for 4 t + 2, + 3).
// Transposed, it hands a lane dims 2 g, 2 g + 1 of tokens 2 t, 2 t + 1; one byte
// permutation puts each dim's tokens side by side, and rows g, g + 8 of the output
// stand for dims 2 g, 2 g + 1.
//
// Precision: a bf16 query head is scaled by a power of two into fp16's range (exact
// down to 2^-31 of its largest element, below that off by 2^-39 of it at most).
// Weights enter the second product as p b / b_ref in two fp16 parts, lifted as in
// weight_range.cuh; the reference (m, b_ref) is the score and scale of the key with
// the largest p b when it was set, m a score itself (weight_range.cuh says why).  Any
// pair with that sum of exponents would do, and where scales lie far apart (blocks of
// zeros beside others) m is one that keeps p, its sum and b / b_ref in fp32's range.
//
// Runs, rings and merge as in decode_pieces_kernel.cuh, with chunks of 32 tokens and
// no runs to take over.
#pragma once

#include "decode_pieces_kernel.cuh"

namespace pkv {

constexpr int kQ8Tokens = 32;                  // tokens per chunk: two halves of 16
// Twelve warps with two chunks each under way.  (With eight and three the issue slots
// were 42 % used, each warp waiting for its own products: 16 MHA contexts of 8K-32K
// 553 us instead of 444, 128 GQA ones of up to 8192 217 instead of 181.)
constexpr int kQ8Warps = 12;
constexpr int kQ8Stages = 2;
constexpr int kQ8StreamHeads = 4;              // kv heads (warps) per stream at most
constexpr int kQ8Threads = 32 * kQ8Warps;
static_assert(kQ8Warps * kQ8Stages == kPieceWarps * kPieceStages, "piece_shared's barriers");
constexpr float kQ8LeastScale = 0x1p-126f;     // fp32's least normal number

// Scores above a reference's m by more than this move it, whatever their values' scale:
// L stays below 2^kQ8Above a token.
constexpr float kQ8Above = 96.f;

struct Q8Params : PieceParams {
    const float* k_scale;      // [num_blocks, n_kv_heads]
    const float* v_scale;
    // decode_q8_short_kernel on chunks (q_start else null)
    const int32_t* q_start;
    int total_q;
    int max_q_len;
    const unsigned char* v_codes;      // the value pool
};

// Two codes each of the low and the high half of w, as packed fp16 (exact).
__device__ __forceinline__ void q8_widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// The 8x8 matrix of 16-bit elements that a warp holds (lane 4 r + c: row r,
// columns 2 c, 2 c + 1), transposed.
__device__ __forceinline__ uint32_t q8_transpose(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Byte mask of the NaN codes (0x7f, 0xff) of a word.
__device__ __forceinline__ uint32_t q8_nans(uint32_t w) {
    return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// Byte offset of 16-byte unit c of token row t in a box of [16 x D] bytes, swizzled
// over D bytes.
template <int D>
__device__ __forceinline__ uint32_t q8_at(int t, int c) {
    return D == 128 ? (uint32_t)(t * 128 + ((c ^ (t & 7)) << 4))
                    : (uint32_t)(t * 64 + ((c ^ ((t >> 1) & 3)) << 4));
}

// Where lane 4 gid + tig finds its head's query among `heads` rows from q on.
template <int D, typename T>
__device__ __forceinline__ const T* q8_head_row(const T* q, int heads, int lane) {
    return q + (size_t)(lane >> 2 < heads ? lane >> 2 : 0) * D;
}

// One kv head's query heads in one warp, lane = 4 gid + tig: queries as B operands
// of head gid; sums of heads 2 tig and 2 tig + 1 (o[j][0], o[j][2]: dims 16 j + 2
// gid, + 1 of the first; o[j][1], o[j][3]: of the second).
template <int D>
struct Q8Heads {
    uint32_t qb[D / 16][2];
    float o[D / 16][4];
    float qf[2];       // score of a unit product at scale 1
    float m[2];        // the reference: a score,
    float lv[2];       // the logarithm of its value scale,
    float rv[2];       // and the weights' lift over that
    float l[2];        // this lane's part of the sum
};

template <int D, typename T>
__device__ __forceinline__ void q8_heads_start(Q8Heads<D>& st, const T* row, bool real,
                                               float scale_log2, int lane) {
    const int tig = lane & 3;
    uint2 w[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
        w[c] = *reinterpret_cast<const uint2*>(row + 16 * c + 4 * tig);
    float back = 1.f;
    if (std::is_same<T, __half>::value) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            st.qb[c][0] = real ? w[c].x : 0u;
            st.qb[c][1] = real ? w[c].y : 0u;
        }
    } else {
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            const float2 a = unpack2<T>(w[c].x), b = unpack2<T>(w[c].y);
            auto take = [&](float x) { top = fabsf(x) < INFINITY ? fmaxf(top, fabsf(x)) : top; };
            take(a.x), take(a.y), take(b.x), take(b.y);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest to 2^14 .. 2^15
        const int e = min(max((int)(__float_as_uint(top) >> 23), 24), 254);
        const float to = __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23);
        back = __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            const float2 a = unpack2<T>(w[c].x), b = unpack2<T>(w[c].y);
            st.qb[c][0] = real ? pack2<__half>(a.x * to, a.y * to) : 0u;
            st.qb[c][1] = real ? pack2<__half>(b.x * to, b.y * to) : 0u;
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        st.qf[e] = scale_log2 * __shfl_sync(0xffffffffu, back, 4 * (2 * tig + e));
        st.m[e] = -INFINITY;
        st.lv[e] = 0.f;
        st.rv[e] = 1.f;
        st.l[e] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) st.o[j][0] = st.o[j][1] = st.o[j][2] = st.o[j][3] = 0.f;
}

// The scales of a chunk's halves (0 and 1 where there is none).
struct Q8Scales {
    float k[2], v[2];
};

// Value scales between which p and b / b_ref stay within fp32's range as they are.
__device__ __forceinline__ bool q8_usual(float b) { return b >= 0x1p-60f && b <= 0x1p16f; }

// min(x, 2^127); NaN stays.
__device__ __forceinline__ float q8_bounded(float x) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(0x1p127f));
    return y;
}

// One chunk: halves of 16 tokens at kbase / vbase (+ 16 D bytes), `valid[h]` of a
// half's tokens inside the context (0: nothing was loaded, or its block is
// missing).  PRECISE: see piece_chunk.  MASKED: of `left[h]` tokens from the half's
// first one on (0 if its block is missing), this lane's heads do not see the last less[e].
// APART: value scales may be any, else those so far and here are q8_usual.
template <int D, bool PRECISE, bool MASKED, bool APART>
__device__ __forceinline__ void q8_chunk_of(Q8Heads<D>& st, uint32_t kbase, uint32_t vbase,
                                         const int (&valid)[2], const int (&left)[2],
                                         const int (&less)[2], const Q8Scales& sc, int lane) {
    using Range = WeightRange<__half>;
    constexpr uint32_t HALF = 16 * D;
    const int gid = lane >> 2, tig = lane & 3;
    const int mat = lane >> 3, mrow = lane & 7;
    // ldmatrix matrices: (tokens 0-7, unit c), (8-15, c), (0-7, c+1), (8-15, c+1)
    const int tok = (mat & 1) * 8 + mrow, unit = mat >> 1;

    // ---- scores: rows = tokens, columns = query heads
    float x[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {
            uint32_t r0, r1, r2, r3;
            ldsm_x4(kbase + h * HALF + q8_at<D>(tok, c + unit), r0, r1, r2, r3);
            uint32_t a[4];
            q8_widen(r0, a[0], a[2]);
            q8_widen(r1, a[1], a[3]);
            mma16816<__half>(s0, a, st.qb[c][0], st.qb[c][1]);
            q8_widen(r2, a[0], a[2]);
            q8_widen(r3, a[1], a[3]);
            mma16816<__half>(s1, a, st.qb[c + 1][0], st.qb[c + 1][1]);
        }
        // this lane: tokens gid (x0, x1) and gid + 8 (x2, x3) of heads 2 tig, + 1
        const float f0 = st.qf[0] * sc.k[h], f1 = st.qf[1] * sc.k[h];
        const int see0 = MASKED ? left[h] - less[0] : valid[h];
        const int see1 = MASKED ? left[h] - less[1] : valid[h];
        x[h][0] = gid < see0 ? __fmul_rn(s0[0] + s1[0], f0) : -INFINITY;
        x[h][1] = gid < see1 ? __fmul_rn(s0[1] + s1[1], f1) : -INFINITY;
        x[h][2] = gid + 8 < see0 ? __fmul_rn(s0[2] + s1[2], f0) : -INFINITY;
        x[h][3] = gid + 8 < see1 ? __fmul_rn(s0[3] + s1[3], f1) : -INFINITY;
    }
    // ---- the reference, where a weight would leave its range
    float lv[2], bv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        bv[h] = fmaxf(sc.v[h], kQ8LeastScale);
        lv[h] = __log2f(bv[h]);
    }
    float top[2][2];
    bool beyond = false;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            top[h][e] = fmaxf(x[h][e], x[h][2 + e]);
            // (apart: the scales' part bounded, so that a score kQ8Above above m is beyond too)
            const float of = lv[h] - st.lv[e];
            beyond |= (top[h][e] - st.m[e]) + (APART ? fmaxf(of, Range::GROW - kQ8Above) : of) >
                      Range::GROW;
        }
    if (__any_sync(0xffffffffu, beyond)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float m = st.m[e], l = st.lv[e], b = 0.f, high = m;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float t = top[h][e];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
                if (t > -INFINITY && (m == -INFINITY || (t - m) + (lv[h] - l) > 0.f)) {
                    m = t;
                    l = lv[h];
                    b = bv[h];
                }
                high = fmaxf(high, t);
            }
            if (b != 0.f || (APART && high - m > kQ8Above)) {
                // lower for a scale below 2^-60, but never below what it was, nor far
                // below a score
                const float to = APART ? fmaxf(fmaxf(m + fminf(l + 60.f, 0.f),
                                                     high - (kQ8Above - 6.f)), st.m[e])
                                       : m;
                l += m - to;
                const float al = st.m[e] == -INFINITY ? 1.f : exp2f(st.m[e] - to);
                const float ao = st.m[e] == -INFINITY ? 1.f : exp2f((st.m[e] - to) + (st.lv[e] - l));
                st.rv[e] = (!APART || (to == m && b != 0.f) ? __frcp_rn(b) : exp2f(-l)) *
                           (1.f / Range::UNLIFT);
                st.m[e] = to;
                st.lv[e] = l;
                st.l[e] *= al;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    st.o[j][e] *= ao;
                    st.o[j][2 + e] *= ao;
                }
            }
        }
    }
    // ---- weights, in two parts, as the B operand (rows = tokens, columns = heads)
    uint32_t hi[2][2], lo[2][2];
    const float mu0 = st.m[0] == -INFINITY ? 0.f : st.m[0];
    const float mu1 = st.m[1] == -INFINITY ? 0.f : st.m[1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float f0 = sc.v[h] * st.rv[0], f1 = sc.v[h] * st.rv[1];
        if (APART) {                       // (where p is next to nothing)
            f0 = q8_bounded(f0);
            f1 = q8_bounded(f1);
        }
        const float p0 = exp2f(x[h][0] - mu0), p1 = exp2f(x[h][1] - mu1);
        const float p2 = exp2f(x[h][2] - mu0), p3 = exp2f(x[h][3] - mu1);
        st.l[0] += p0 + p2;
        st.l[1] += p1 + p3;
        // (a half with nothing in it may have any scale)
        const bool any0 = (MASKED ? left[h] - less[0] : valid[h]) > 0;
        const bool any1 = (MASKED ? left[h] - less[1] : valid[h]) > 0;
        const float w0 = any0 ? p0 * f0 : 0.f, w1 = any1 ? p1 * f1 : 0.f;
        const float w2 = any0 ? p2 * f0 : 0.f, w3 = any1 ? p3 * f1 : 0.f;
        const uint32_t a = pack2<__half>(w0, w1), b = pack2<__half>(w2, w3);
        const float2 fa = unpack2<__half>(a), fb = unpack2<__half>(b);
        hi[h][0] = q8_transpose(a);
        hi[h][1] = q8_transpose(b);
        lo[h][0] = q8_transpose(pack2<__half>(w0 - fa.x, w1 - fa.y));
        lo[h][1] = q8_transpose(pack2<__half>(w2 - fb.x, w3 - fb.y));
    }
    // ---- O^T += V^T P^T; rows behind the context may hold NaN: cleared
    // (a byte permutation's result: tokens 2 tig, 2 tig + 1 of one dim, then of the next)
    uint32_t vm[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k)
            vm[h][k] = (8 * k + 2 * tig < valid[h] ? 0x00ff00ffu : 0u) |
                       (8 * k + 2 * tig + 1 < valid[h] ? 0xff00ff00u : 0u);
#pragma unroll
    for (int c = 0; c < D / 16; c += 2) {
        float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t r[4];
            ldsm_x4_trans(vbase + h * HALF + q8_at<D>(tok, c + unit), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t a[4];
                q8_widen(__byte_perm(r[2 * u], 0u, 0x3120) & vm[h][0], a[0], a[1]);
                q8_widen(__byte_perm(r[2 * u + 1], 0u, 0x3120) & vm[h][1], a[2], a[3]);
                float(&d)[4] = PRECISE ? acc[u] : st.o[c + u];
                mma16816<__half>(d, a, lo[h][0], lo[h][1]);
                mma16816<__half>(d, a, hi[h][0], hi[h][1]);
            }
        }
        if (PRECISE)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) st.o[c + u][e] += acc[u][e];
    }
}

// With the usual scales nothing leaves fp32's range; `apart` says whether there have been
// others among a piece's chunks so far (the same for all lanes).
template <int D, bool PRECISE, bool MASKED = false>
__device__ __forceinline__ void q8_chunk(Q8Heads<D>& st, uint32_t kbase, uint32_t vbase,
                                         const int (&valid)[2], const int (&left)[2],
                                         const int (&less)[2], const Q8Scales& sc, bool& apart,
                                         int lane) {
    apart |= !q8_usual(sc.v[0]) || !q8_usual(sc.v[1]);
    if (apart)
        q8_chunk_of<D, PRECISE, MASKED, true>(st, kbase, vbase, valid, left, less, sc, lane);
    else
        q8_chunk_of<D, PRECISE, MASKED, false>(st, kbase, vbase, valid, left, less, sc, lane);
}

// A piece's result: the normalised rows row_of(head) of `heads` heads to the output
// (WHOLE) or, with (m, L), to o and ml (of the workspace or shared memory).
template <int D, bool WHOLE, class RowOf>
__device__ __forceinline__ void q8_store(const Q8Heads<D>& st, const Q8Params& p, int heads,
                                         RowOf row_of, float* o, float* ml, int lane) {
    const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float l = st.l[e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        const int hh = 2 * tig + e;
        if (hh >= heads) continue;
        // (in two factors: either alone may leave fp32's range)
        const float inv = l != 0.f ? __frcp_rn(l) : 0.f;
        const float b = __frcp_rn(st.rv[e]);
        const size_t row = row_of(hh);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const float v0 = st.o[j][e] * inv * b, v1 = st.o[j][2 + e] * inv * b;
            const size_t at = row * D + 16 * j + 2 * gid;
            if (!WHOLE)
                *reinterpret_cast<float2*>(o + at) = make_float2(v0, v1);
            else if (p.out_dtype == PKV_F32)
                *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.out) + at) =
                    make_float2(v0, v1);
            else
                *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.out) + at) =
                    pack_out(v0, v1, p.out_dtype);
        }
        if (!WHOLE && gid == 0)
            *reinterpret_cast<float2*>(ml + row * 2) = make_float2(st.m[e], l);
    }
}

// A half chunk's K and V rows (a box of [16 x D] bytes each).
__device__ __forceinline__ void q8_load(uint32_t k, const CUtensorMap* tm_k, uint32_t v,
                                        const CUtensorMap* tm_v, uint32_t bar, int row, int head,
                                        int block, uint64_t policy, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %9, 0;\n\t"
        "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%10, %5, %6, %7}], [%4], %8;\n\t"
        "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%2], [%3, {%10, %5, %6, %7}], [%4], %8;\n\t}" ::"r"(k),
        "l"(reinterpret_cast<uint64_t>(tm_k)), "r"(v), "l"(reinterpret_cast<uint64_t>(tm_v)),
        "r"(bar), "r"(row), "r"(head), "r"(block), "l"(policy), "r"(lead), "r"(0)
        : "memory");
}

// Bytes of the control area beside piece_shared's: the block of each half of the
// chunks in the rings.
constexpr size_t kQ8BlockBytes = (size_t)kQ8Warps * kQ8Stages * 2 * sizeof(int);

// One warp's work on the CTA's runs (piece_worker's, on 8-bit pages).
template <int D, typename T, bool PRECISE>
__device__ __forceinline__ void q8_worker(const Q8Params& p, const CUtensorMap& tm_k,
                                          const CUtensorMap& tm_v, const PieceShared& sh,
                                          int* blocks, const PieceRuns& runs) {
    constexpr uint32_t HALF = 16 * D;                 // half a chunk of K (or V)
    constexpr uint32_t SLOT = 4 * HALF;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int HW = p.stream_heads, hw = warp % HW;
    unsigned char* ring = sh.ring + (size_t)warp * kQ8Stages * SLOT;
    uint64_t* full = sh.bars + warp * kQ8Stages;
    int* slot_block = blocks + warp * kQ8Stages * 2;
    const int pages = kQ8Tokens / p.block_size;       // of a chunk: 2 or 1
    const uint64_t policy = l2_policy_evict_first();
    const uint32_t lead = lane == 0 ? 1u : 0u;
    if (lane == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }

    const int v = piece_stream(p, runs, blockIdx.x, warp, kQ8Warps);
    if (v < 0) return;
    PieceCursor ld = piece_locate<true, kQ8Tokens>(p, sh, runs, v, lane);   // the next to load
    PieceCursor at = ld;                                                    // and to work on
    int win = -1, bid = -1;      // block ids of the pair's pages win .. win + 31

    auto issue = [&](int st) {
        const int page0 = ld.c * pages;
        const int kvh = ld.hg * HW + hw;
        if (win < 0 || page0 < win || page0 + pages > win + 32) {
            win = page0;
            const int page = win + lane;
            const bool want = page * p.block_size < ld.n && page < p.max_blocks_per_seq;
            bid = want ? p.block_tables[(size_t)ld.s * p.max_blocks_per_seq + page] : -1;
            if (want && (bid < 0 || bid >= p.num_blocks)) {
                raise_error(p.errors, PKV_DEVERR_BLOCK_ID);
                bid = -1;
            }
            // the scales come to L2 with their pages
            if (bid >= 0) {
                const size_t i = (size_t)bid * p.n_kv_heads + kvh;
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.k_scale + i));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.v_scale + i));
            }
        }
        int b[2];
        b[0] = __shfl_sync(0xffffffffu, bid, page0 - win);
        b[1] = __shfl_sync(0xffffffffu, bid, page0 + pages - 1 - win);
        if (ld.c * kQ8Tokens + 16 >= ld.n) b[1] = -1;      // nothing in the second half
        const int loads = (b[0] >= 0) + (b[1] >= 0);
        const uint32_t dst = smem_addr(ring) + st * SLOT, bar = smem_addr(&full[st]);
        if (lane == 0) {
            slot_block[2 * st] = b[0];
            slot_block[2 * st + 1] = b[1];
            if (loads)
                mbar_arrive_expect_tx(&full[st], loads * 2 * HALF);
            else
                mbar_arrive(&full[st]);
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (b[h] >= 0)
                q8_load(dst + h * HALF, &tm_k, dst + (2 + h) * HALF, &tm_v, bar,
                        pages == 1 ? 16 * h : 0, kvh, b[h], policy, lead);
        const int s = ld.s, hg = ld.hg;
        piece_advance<true, kQ8Tokens>(p, sh, ld);
        if (ld.s != s || ld.hg != hg) win = -1;
    };

    Q8Heads<D> state;
    bool fresh = true;                 // the next chunk starts a piece
    bool from_start = false;           // the piece holds the pair's first chunk
    bool apart = false;                // its scales so far are not all q8_usual
    int st = 0, put = 0, in_flight = 0;
    uint32_t phase = 0;
    for (;;) {
        // ---- keep the ring full
        while (in_flight < kQ8Stages && ld.left > 0) {
            issue(put);
            if (++put == kQ8Stages) put = 0;
            ++in_flight;
        }
        if (in_flight == 0) break;
        // ---- one chunk
        const int kvh = at.hg * HW + hw, qh0 = kvh * p.group;
        Q8Scales sc;
        int valid[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int b = slot_block[2 * st + h];
            const size_t i = (size_t)max(b, 0) * p.n_kv_heads + kvh;
            valid[h] = b >= 0 ? min(16, at.n - at.c * kQ8Tokens - 16 * h) : 0;
            sc.k[h] = b >= 0 ? __ldg(p.k_scale + i) : 0.f;
            sc.v[h] = b >= 0 ? __ldg(p.v_scale + i) : 1.f;
        }
        if (fresh) {
            q8_heads_start<D, T>(state,
                                 q8_head_row<D, T>(reinterpret_cast<const T*>(p.q) +
                                                       ((size_t)at.s * p.n_heads + qh0) * D,
                                                   p.group, lane),
                                 lane >> 2 < p.group, p.scale_log2, lane);
            from_start = at.c == at.first;
            fresh = false;
            apart = false;
        }
        const bool w = mbar_wait(&full[st], phase, p.errors);
        if (!__all_sync(0xffffffffu, w)) {
            // the loads still in flight land before the CTA may exit
            for (; in_flight > 0; --in_flight) {
                mbar_wait(&full[st], phase, p.errors);
                if (++st == kQ8Stages) {
                    st = 0;
                    phase ^= 1u;
                }
            }
            break;
        }
        const uint32_t kbase = smem_addr(ring) + st * SLOT;
        if (valid[0] > 0 || valid[1] > 0)
            q8_chunk<D, PRECISE>(state, kbase, kbase + 2 * HALF, valid, valid, valid, sc, apart,
                                 lane);
        __syncwarp();
        --in_flight;
        if (++st == kQ8Stages) {
            st = 0;
            phase ^= 1u;
        }
        // ---- the piece ends with the pair or with the run
        const bool pair_end = at.c + 1 == at.end;
        if (pair_end || at.left == 1) {
            const size_t pair = (size_t)at.s * p.n_kv_heads + kvh;
            const size_t own = (size_t)at.s * p.n_heads + qh0;
            if (from_start && pair_end)
                q8_store<D, true>(
                    state, p, p.group, [&](int h) { return own + h; }, nullptr, nullptr, lane);
            else {
                const size_t to = from_start ? own
                                             : (size_t)p.num_seqs * p.n_heads +
                                                   ((size_t)at.v * HW + hw) * p.group;
                q8_store<D, false>(
                    state, p, p.group, [&](int h) { return to + h; }, p.ws_o, p.ws_ml, lane);
            }
            if (lane == 0) {
                if (from_start) p.seg_first[pair] = at.v;
                if (pair_end) p.seg_last[pair] = at.v;
            }
            fresh = true;
        }
        piece_advance<true, kQ8Tokens>(p, sh, at);
    }
}

inline size_t decode_q8_smem_bytes(int D) {
    return decode_pieces_smem_bytes(D) + kQ8BlockBytes;
}

// A run of equal length for each stream (short runs that CTAs take over, as in
// decode_pieces_kernel, need one warp more, whose registers the twelve cannot spare:
// 128 a thread spill, 662 us instead of 444 for 16 contexts of 8K-32K tokens).
template <int D, typename T, bool PRECISE>
__global__ void __launch_bounds__(kQ8Threads, 1)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ Q8Params p) {
    launch_dependents();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char* sm = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    unsigned char* control = sm + decode_pieces_ring_bytes(D);
    int* blocks = reinterpret_cast<int*>(control + 64);
    PieceShared sh = piece_shared(sm, control + 64 + kQ8BlockBytes);
    if (threadIdx.x < kPieceThreads) piece_plan<true, kQ8Tokens>(p, sh);
    __syncthreads();
    const int chunks = sh.cum[(p.num_seqs + 255) / 256];
    q8_worker<D, T, PRECISE>(p, tm_k, tm_v, sh, blocks, piece_runs(p, chunks, kQ8Warps));
}

// Short contexts: a CTA per (sequence, kv head), its warps taking the chunks in
// turn, their states merged in shared memory: one launch, and no line of units to
// lay out first.
// CHUNK: sequence s has the queries q_start[s] .. q_start[s + 1] - 1, and 8 / G tokens of
// it (the blockIdx.z-th) with their G heads are the product's eight columns.  The last
// tokens of the context that some of them do not see are masked in the scores; NaN in
// their values is taken out in shared memory and put where it belongs at the end.
constexpr int kQ8ShortWarps = 12;        // at most

inline size_t decode_q8_short_smem_bytes(int D, int warps) {
    return 1024 + (size_t)warps * kQ8Stages * 4 * 16 * D;
}

template <int D, typename T, bool PRECISE, bool CHUNK>
__global__ void __launch_bounds__(32 * kQ8ShortWarps)
    decode_q8_short_kernel(const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ Q8Params p) {
    constexpr uint32_t HALF = 16 * D, SLOT = 4 * HALF;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ uint64_t s_bar[kQ8ShortWarps * kQ8Stages];
    __shared__ float s_ml[kQ8ShortWarps * 8 * 2];
    __shared__ int s_poison;
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char* sm = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int kvh = blockIdx.x, s = blockIdx.y, qh0 = kvh * p.group;
    unsigned char* ring = sm + (size_t)warp * kQ8Stages * SLOT;
    uint64_t* full = s_bar + warp * kQ8Stages;
    const int raw_n = p.context_lens[s];
    int n = piece_length(p, s);
    size_t row0 = (size_t)s * p.n_heads + qh0;       // of the first column
    int tokens = 1;                                  // whose heads are the columns
    bool ok = raw_n == n;
    if (CHUNK) {
        const int qs0 = p.q_start[s], qs1 = p.q_start[s + 1], q_len = qs1 - qs0;
        const int first = (int)blockIdx.z * (8 / p.group);
        ok = ok && q_len >= 0 && q_len <= n && qs0 >= 0 && qs1 <= p.total_q && q_len <= p.max_q_len;
        tokens = min(8 / p.group, q_len - first);
        n -= q_len - first - tokens;                 // the last one's context
        row0 += (size_t)(qs0 + first - s) * p.n_heads;
    }
    if (!ok && threadIdx.x == 0 && kvh == 0 && blockIdx.z == 0)
        raise_error(p.errors, PKV_DEVERR_CONTEXT);
    if (CHUNK && (!ok || tokens <= 0)) return;
    const int cols = tokens * p.group;
    auto row_of = [&](int c) -> size_t {
        return CHUNK ? row0 + (size_t)(c / p.group) * p.n_heads + c % p.group : row0 + c;
    };
    // tokens of the context that column c does not see, the last ones
    auto hidden = [&](int c) { return CHUNK ? max(tokens - 1 - c / p.group, 0) : 0; };
    const int less[2] = {hidden(2 * (lane & 3)), hidden(2 * (lane & 3) + 1)};
    if (CHUNK) {
        if (threadIdx.x == 0) s_poison = 0;
        __syncthreads();
    }
    const int chunks = (n + kQ8Tokens - 1) / kQ8Tokens;
    if (lane == 0) {
        for (int i = 0; i < kQ8Stages; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
    }
    __syncwarp();
    const uint64_t policy = l2_policy_evict_first();
    const uint32_t lead = lane == 0 ? 1u : 0u;
    // halves of chunk c: their blocks (-1: none), their loads started
    struct Blocks {
        int b[2];
        Q8Scales sc;
    };
    auto issue = [&](int c, int st) -> Blocks {
        Blocks r;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int t = c * kQ8Tokens + 16 * h;
            r.b[h] = -1;
            r.sc.k[h] = 0.f;
            r.sc.v[h] = 1.f;
            if (t >= n) continue;
            const int b =
                __ldg(p.block_tables + (size_t)s * p.max_blocks_per_seq + t / p.block_size);
            if (b < 0 || b >= p.num_blocks) {
                raise_error(p.errors, PKV_DEVERR_BLOCK_ID);
                continue;
            }
            r.b[h] = b;
            const size_t i = (size_t)b * p.n_kv_heads + kvh;
            r.sc.k[h] = __ldg(p.k_scale + i);
            r.sc.v[h] = __ldg(p.v_scale + i);
        }
        const int loads = (r.b[0] >= 0) + (r.b[1] >= 0);
        if (lane == 0) {
            if (loads)
                mbar_arrive_expect_tx(&full[st], loads * 2 * HALF);
            else
                mbar_arrive(&full[st]);
        }
        __syncwarp();
        const uint32_t dst = smem_addr(ring) + st * SLOT;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (r.b[h] >= 0)
                q8_load(dst + h * HALF, &tm_k, dst + (2 + h) * HALF, &tm_v, smem_addr(&full[st]),
                        (c * kQ8Tokens + 16 * h) % p.block_size, kvh, r.b[h], policy, lead);
        return r;
    };
    Q8Heads<D> state;
    if (warp < chunks) {
        Blocks now = issue(warp, 0);
        const int own = lane >> 2;
        q8_heads_start<D, T>(state,
                             reinterpret_cast<const T*>(p.q) + row_of(own < cols ? own : 0) * D,
                             own < cols, p.scale_log2, lane);
        int st = 0;
        uint32_t phase = 0;
        bool apart = false;
        for (int c = warp; c < chunks; c += warps) {
            Blocks next = now;
            const bool more = c + warps < chunks;
            if (more) next = issue(c + warps, st ^ 1);
            const bool w = mbar_wait(&full[st], phase, p.errors);
            if (!__all_sync(0xffffffffu, w)) {
                // the loads still in flight land before the CTA may exit
                mbar_wait(&full[st], phase, p.errors);
                if (more) mbar_wait(&full[st ^ 1], st ? phase ^ 1u : phase, p.errors);
                break;
            }
            int valid[2], left[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                left[h] = now.b[h] >= 0 ? n - c * kQ8Tokens - 16 * h : 0;
                valid[h] = min(16, left[h]);
            }
            const uint32_t kbase = smem_addr(ring) + st * SLOT;
            if (CHUNK) {
                // (a lane has 16 bytes of a row; nothing is loaded over the context's last
                // chunks again)
                const int to = min(n, (c + 1) * kQ8Tokens);
                for (int k = max(n - tokens + 1, c * kQ8Tokens); k < to; ++k) {
                    const int h = k / 16 % 2;
                    if ((h ? now.b[1] : now.b[0]) < 0 || lane >= D / 16) continue;
                    uint4* unit = reinterpret_cast<uint4*>(ring + st * SLOT + (2 + h) * HALF +
                                                           q8_at<D>(k % 16, lane));
                    const uint4 w = *unit;
                    const uint4 bad = make_uint4(q8_nans(w.x), q8_nans(w.y), q8_nans(w.z),
                                                 q8_nans(w.w));
                    if ((bad.x | bad.y | bad.z | bad.w) == 0u) continue;
                    *unit = make_uint4(w.x & ~bad.x, w.y & ~bad.y, w.z & ~bad.z, w.w & ~bad.w);
                    s_poison = 1;
                }
                __syncwarp();
            }
            if (valid[0] > 0 || valid[1] > 0)
                q8_chunk<D, PRECISE, CHUNK>(state, kbase, kbase + 2 * HALF, valid, left, less,
                                            now.sc, apart, lane);
            __syncwarp();
            now = next;
            if (st) phase ^= 1u;
            st ^= 1;
        }
    }
    // ---- the warps' states (each over its own ring)
    const int active = min(chunks, warps);
    if (!CHUNK && active == 1) {
        if (warp == 0) q8_store<D, true>(state, p, cols, row_of, nullptr, nullptr, lane);
        return;
    }
    if (warp < active)
        q8_store<D, false>(
            state, p, cols, [](int c) { return (size_t)c; }, reinterpret_cast<float*>(ring),
            s_ml + warp * 16, lane);
    __syncthreads();
    for (int e = threadIdx.x; e < cols * (D / 2); e += blockDim.x) {
        const int h = e / (D / 2), d = e % (D / 2) * 2;
        float2 ml = make_float2(-INFINITY, 0.f);
        for (int w = 0; w < active; ++w)
            ml = join_ml(ml, *reinterpret_cast<const float2*>(s_ml + w * 16 + 2 * h));
        const float inv = ml.y != 0.f ? 1.f / ml.y : 0.f;
        float2 o = make_float2(0.f, 0.f);
        for (int w = 0; w < active; ++w) {
            const float2 a = *reinterpret_cast<const float2*>(s_ml + w * 16 + 2 * h);
            const float f = a.y != 0.f ? a.y * exp2f(a.x - ml.x) * inv : 0.f;
            const float2 x = *reinterpret_cast<const float2*>(
                sm + (size_t)w * kQ8Stages * SLOT + (h * D + d) * sizeof(float));
            o.x += f * x.x;
            o.y += f * x.y;
        }
        if (CHUNK && s_poison) {
            // NaN that was taken out, to the columns that see it
            for (int k = n - tokens + 1; k < n - hidden(h); ++k) {
                const int b = p.block_tables[(size_t)s * p.max_blocks_per_seq + k / p.block_size];
                if (b < 0 || b >= p.num_blocks) continue;
                const size_t row = (size_t)b * p.block_size + k % p.block_size;
                const unsigned char* v = p.v_codes + (row * p.n_kv_heads + kvh) * D + d;
                if ((v[0] & 0x7f) == 0x7f) o.x = NAN;
                if ((v[1] & 0x7f) == 0x7f) o.y = NAN;
            }
        }
        const size_t at = row_of(h) * D + d;
        if (p.out_dtype == PKV_F32)
            *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.out) + at) = o;
        else
            *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.out) + at) =
                pack_out(o.x, o.y, p.out_dtype);
    }
}

// Rows cut into pieces, merged; rows of no token, zero.  Grid x: rows of a
// sequence, kFinishWarps / W per CTA; y: sequences.
template <int D, int W>
__global__ void __launch_bounds__(kFinishThreads)
    decode_q8_finish_kernel(const __grid_constant__ PieceParams p) {
    __shared__ __align__(16) float s_o[kFinishWarps * D];
    dependency_wait();
    const int s = blockIdx.y, h = blockIdx.x * (kFinishWarps / W) + (threadIdx.x >> 5) / W;
    const PieceSet c = piece_set(p, s, min(h, p.n_heads - 1), piece_length(p, s), 0);
    merge_rows<D, W>(p, c, h < p.n_heads && (c.extra || !c.first), s, h, s_o);
}

}  // namespace pkv
