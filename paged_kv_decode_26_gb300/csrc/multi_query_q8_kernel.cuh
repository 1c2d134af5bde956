// multi_query_q8_kernel.cuh -- causal attention of several new tokens per
// sequence over 8-bit pages (e4m3 with a scale per block and kv head) on tcgen05
// (sm_103a): paged_attn_multi_query_q8.
//
// Mathematics: with codes k_t, v_t and the scales a_t, b_t of token t's block,
// scores x_t = scale log2(e) a_t (q . k_t), weights w_t = 2^(x_t - M) b_t, O = sum
// w_t v_t and L = sum w_t / b_t; the result is O / L.
//
// Tiles: 128 rows are 128 / G query tokens x the G query heads of a kv head; a CTA
// has two row tiles (256 rows) that share every key tile of 128 keys: while the
// softmax of one runs, the tensor core multiplies for the other.
// Codes are exact in fp16, so both products are fp16 ones: warps 9-15 widen the
// codes of K and V on their way from global to shared memory, 16 keys at a time in
// turn, the next ones already in registers (no copy of the codes in shared memory:
// the products' operands take most of its bandwidth).  Queries become fp16 too, each row
// scaled by a power of two (exact down to 2^-31 of the row's largest element, below
// that off by 2^-39 of it at most).
// A block's scales are one number per 16 keys: a_t multiplies the exponent's
// factor, log2 b_t joins its addend, so they cost nothing per element; the sum L
// takes the weights of 16 keys times 1 / b_t.
//
// Roles: warps 0-3 and 4-7 the softmax of tile 0 and 1, a thread per row; warp 8
// issues every MMA; 9-15 load and widen K and V.
//
// Measured: 2 chunks of 2048 tokens behind 12K-16K, 32 heads of 128, 844 us (1.16
// PFLOP/s, 0.61 of a library bf16 product's rate), fp32 outputs 980-1050; 8 of 100-512
// tokens at 1K-8K, 32 query and 8 kv heads, 158-163 us, fp32 outputs 200.  (Value scales
// far apart, handled where they occur, cost 0.5-0.8 % of this.)  A step of 128 keys takes 3500 cycles, of which the tensor core
// needs 2050 and the operands' way through shared memory as many; the rest is the
// softmax's chain (scores in, maximum, weights out), two row tiles being all that the
// tensor memory holds.  Without the exponentials it would be 8 % faster, without loads
// and widening 14 %.  Codes through shared memory by TMA: the same; two issuing warps 990
// us instead of 871; weights by the old maximum beside the new one 906.  One CTA per SM
// on an equal share of all key tiles 890 instead of 840 (160 -> 213 us for the
// grouped heads): neighbours no longer read a head's keys at the same time.
//
// Precision: S, M, L and O are fp32.  A weight is rounded once to fp16 before the
// second product (fp32 outputs: two parts), lifted and bounded as in
// weight_range.cuh; M = m + lb with m the score and lb = log2 b_ref of the key with the
// largest weight when it was set, or their sum and 0 (m has to be a score itself only
// where scores are large), and L is kept relative to 2^m.  Value scales outside 2^-60
// .. 2^16 (blocks of zeros have the least), or a reference of such, take a way of
// their own, where L has its own exponentials: weights there may be far below or
// above what they add to L.  O accumulates in the tensor core, which drops what lies
// below its last bit: up to 2^-23 of O per 16 keys.
#pragma once

#include "attn_tc_kernel.cuh"
#include "decode_q8_kernel.cuh"

namespace pkv {

constexpr int kMq8Keys = 128;
constexpr int kMq8Rows = 128;
constexpr int kMq8Threads = 512;      // 8 softmax warps, 1 MMA, 7 that widen
constexpr int kMq8Widen = 7;
// Registers per thread: 512 x 128 at launch
constexpr int kMq8SoftmaxRegs = 184, kMq8OtherRegs = 72;
static_assert(256 * kMq8SoftmaxRegs + 256 * kMq8OtherRegs <= kMq8Threads * 128, "registers");
// Key tiles whose scales are kept: K of tile j + STAGES / 2 is widened as soon as
// S_j is formed, while its softmax still reads the scales of tile j.
constexpr int kMq8Scales = 8;

struct Mq8Params : MultiQueryParams {
    const void* k_pool;
    const void* v_pool;
    const float* k_scale;
    const float* v_scale;
    int q_bf16;
    // Items are pairs of row tiles of a kv head, `tiles` of them for every sequence and
    // head: a CTA for each of the first `whole`, and for each of the others one for every
    // of `splits` parts of its keys
    int tiles;
    int whole;
    int splits;
    int block_size;
    float* part_o;             // [others, splits, 256 rows, D], normalised
    float* part_ml;            // [others, splits, 256 rows, 2]
    int4* heads;               // [others]: sequence (-1: nothing to merge), kv head, pair of
                               // row tiles, parts with keys
};

// log2 of value scales for which w_t / b_t adds up to L as it is.
constexpr float kMq8LeastLog = -60.f, kMq8MostLog = 16.f;
__device__ __forceinline__ bool mq8_usual(float lb) {
    return lb >= kMq8LeastLog && lb <= kMq8MostLog;
}
// Scores above m by more than this move it, whatever their values' scale.
constexpr float kMq8Above = 64.f;

// Of a key tile's groups of 16 keys: a, log2 b and 1 / b, and whether there is a page.
struct __align__(16) Mq8Scale {
    float a[8], lb[8], ib[8];
    unsigned char page[16];            // 8 of them: 0: none, 1, or 2: b not mq8_usual
};

template <int D>
struct Mq8Sizes {
    static constexpr int HALVES = D / 64;
    static constexpr uint32_t KV_HALF = kMq8Keys * 128;
    static constexpr uint32_t KV_BYTES = HALVES * KV_HALF;     // a widened K or V tile
    static constexpr uint32_t Q_HALF = kMq8Rows * 128;
    static constexpr uint32_t Q_BYTES = HALVES * Q_HALF;
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr uint32_t TILE_COLS = 256;                 // per row tile: O, then S / P
    static constexpr uint32_t S_COL = D;
    static_assert(STAGES / 2 < kMq8Scales, "scales");
    static constexpr size_t SMEM = 1024 + 2 * Q_BYTES + STAGES * KV_BYTES +
                                   kMq8Scales * sizeof(Mq8Scale) + (2 * STAGES + 12) * 8 + 16;
};

// 16 codes to two chunks of 8 fp16.
__device__ __forceinline__ void mq8_widen(const uint4& w, uint4& a, uint4& b) {
    q8_widen(w.x, a.x, a.y);
    q8_widen(w.y, a.z, a.w);
    q8_widen(w.z, b.x, b.y);
    q8_widen(w.w, b.z, b.w);
}

// 16 bytes that nothing on this SM reads again.
__device__ __forceinline__ uint4 mq8_load(const void* p) {
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p));
    return v;
}

__device__ __forceinline__ void mq8_store(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

// Rows of items in pieces, merged: a warp per row of the x-th item of several parts.
constexpr int kMq8MergeRows = 16;
constexpr int kMq8MergeThreads = 32 * kMq8MergeRows;
template <int D>
__global__ void __launch_bounds__(kMq8MergeThreads)
    multi_query_q8_merge_kernel(const __grid_constant__ Mq8Params p) {
    constexpr int V = D / 32;
    dependency_wait();
    const int4 head = p.heads[blockIdx.x];
    if (head.x < 0) return;
    const int lane = threadIdx.x & 31, G = p.group, QT = kMq8Rows / G;
    const int pieces = head.w;
    const int qs0 = p.q_start[head.x] + head.z * 2 * QT;
    const int rows = min(p.q_start[head.x + 1] - qs0, 2 * QT);
    const int i = blockIdx.y * kMq8MergeRows + (threadIdx.x >> 5), tok = i / G;
    if (tok >= rows) return;
    auto row_of = [&](int piece) -> size_t {
        return ((size_t)blockIdx.x * p.splits + piece) * 2 * kMq8Rows + i;
    };
    float2 ml = make_float2(-INFINITY, 0.f);
    for (int w = lane; w < pieces; w += 32)
        ml = join_ml(ml, *reinterpret_cast<const float2*>(p.part_ml + 2 * row_of(w)));
#pragma unroll
    for (int off = 16; off; off /= 2)
        ml = join_ml(ml, make_float2(__shfl_xor_sync(0xffffffffu, ml.x, off),
                                     __shfl_xor_sync(0xffffffffu, ml.y, off)));
    const float inv = ml.y != 0.f ? 1.f / ml.y : 0.f;
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
    for (int w = 0; w < pieces; ++w) {
        const float2 a = *reinterpret_cast<const float2*>(p.part_ml + 2 * row_of(w));
        if (a.y == 0.f) continue;                  // (nothing was written for it)
        const float f = a.y * exp2f(a.x - ml.x) * inv;
        const float* row = p.part_o + row_of(w) * D + lane * V;
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 x = *reinterpret_cast<const float2*>(row + e);
            o[e] += f * x.x;
            o[e + 1] += f * x.y;
        }
    }
    const size_t at =
        ((size_t)(qs0 + tok) * p.n_heads + head.y * G + i % G) * D + lane * V;
#pragma unroll
    for (int e = 0; e < V; e += 2) {
        if (p.out_dtype == PKV_F32)
            *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.out) + at + e) =
                make_float2(o[e], o[e + 1]);
        else
            *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.out) + at + e) =
                pack_out(o[e], o[e + 1], p.out_dtype);
    }
}

template <int D, int BS, int PARTS>
__global__ void __launch_bounds__(kMq8Threads, 1)
    multi_query_q8_kernel(const __grid_constant__ Mq8Params p) {
    using Z = Mq8Sizes<D>;
    using Range = WeightRange<__half>;
    constexpr int STAGES = Z::STAGES;
    constexpr int kParts = 2 * Z::HALVES;          // 16-byte parts of 16 keys' codes per lane
    launch_dependents();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char* sm = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    unsigned char* sQ = sm;
    unsigned char* sKV = sQ + 2 * Z::Q_BYTES;
    Mq8Scale* s_scale = reinterpret_cast<Mq8Scale*>(sKV + STAGES * Z::KV_BYTES);
    uint64_t* kv_full = reinterpret_cast<uint64_t*>(s_scale + kMq8Scales);
    uint64_t* kv_free = kv_full + STAGES;
    uint64_t* q_full = kv_free + STAGES;          // [tile]
    uint64_t* s_full = q_full + 2;
    uint64_t* p_full = s_full + 2;                // [tile][half of the keys]
    uint64_t* o_full = p_full + 4;
    uint64_t* fin = o_full + 2;
    int* s_tmem = reinterpret_cast<int*>(fin + 2);
    int* s_poison = s_tmem + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int cta = blockIdx.x;
    const bool cut = cta >= p.whole && p.splits > 1;
    const int other = cut ? (cta - p.whole) / p.splits : 0;
    const int part = cut ? (cta - p.whole) % p.splits : 0, parts = cut ? p.splits : 1;
    const int item = cut ? p.whole + other : cta;
    int tile = item % p.tiles, kvh = item / p.tiles % p.n_kv_heads,
        s = item / (p.tiles * p.n_kv_heads);
    if (p.lpt_seqs > 0) {
        longest_first(p, reinterpret_cast<int*>(sKV), item, p.tiles, p.n_kv_heads, tile, kvh,
                      s);                               // (sKV: not yet in use)
        __syncthreads();
    }
    const int G = p.group, QT = kMq8Rows / G;
    const int qs0 = p.q_start[s], qs1 = p.q_start[s + 1];
    const int n = p.context_lens[s];
    const int q_len = qs1 - qs0;
    const int tok_lo = tile * 2 * QT;
    const bool bad = q_len < 0 || q_len > n || qs0 < 0 || qs1 > p.total_q ||
                     q_len > p.max_q_len || n > (long long)p.max_pages * BS ||
                     n > (long long)p.max_blocks_per_seq * BS;
    if (bad || tok_lo >= q_len) {
        if (bad && tile == 0 && part == 0 && kvh == 0 && threadIdx.x == 0)
            raise_error(p.errors, PKV_DEVERR_CONTEXT);
        if (cut && part == 0 && threadIdx.x == 0) p.heads[other] = make_int4(-1, 0, 0, 0);
        return;
    }
    const int pos0 = n - q_len + tok_lo;             // position of row tile 0's first token
    const int rows = min(q_len - tok_lo, 2 * QT);    // tokens of this CTA
    const int n_keys = pos0 + rows;                  // keys that some row sees
    // key tiles that the row tiles see, and of them those of this part: j0 + 0, 1, ..
    const int see0 = (pos0 + min(rows, QT) + kMq8Keys - 1) / kMq8Keys;
    const int see1 = rows > QT ? (n_keys + kMq8Keys - 1) / kMq8Keys : 0;
    const int see = max(see0, see1), part_tiles = (see + parts - 1) / parts;
    if (cut && part == 0 && threadIdx.x == 0)
        p.heads[other] = make_int4(s, kvh, tile, (see + part_tiles - 1) / part_tiles);
    const int j0 = part * part_tiles;
    const int nt0 = min(max(see0 - j0, 0), part_tiles), nt1 = min(max(see1 - j0, 0), part_tiles);
    const int n_tiles = max(nt0, nt1);
    if (n_tiles == 0) return;
    // row r of row tile t of this part
    auto unit_of = [&](int t, int r) -> size_t {
        return (((size_t)other * parts + part) * 2 + t) * kMq8Rows + r;
    };

    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(s_tmem)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&kv_full[i], 8);
            mbar_init(&kv_free[i], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&q_full[t], 4);
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[2 * t], 4);
            mbar_init(&p_full[2 * t + 1], 4);
            mbar_init(&o_full[t], 1);
            mbar_init(&fin[t], 1);
        }
        *s_poison = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)*s_tmem;

    if (warp >= 8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMq8OtherRegs));
      if (warp == 8) {
        // ================= every MMA =================
        const uint32_t id_s = tc_idesc<__half>(kMq8Rows, kMq8Keys, 0);
        const uint32_t id_o = tc_idesc<__half>(kMq8Rows, D, 1);
        const uint64_t dq0 = tc_desc_sw128(smem_addr(sQ), 16, 1024);
        const uint64_t dk0 = tc_desc_sw128(smem_addr(sKV), 16, 1024);
        const uint64_t dv0 = tc_desc_sw128(smem_addr(sKV), Z::KV_HALF, 1024);
        const uint32_t lead = elect_one() ? 1u : 0u;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, p.errors));
        };
        // operand i of the ring (K_0, V_0, K_1, V_1, ...)
        auto slot = [&](int i) { return i % STAGES; };
        auto round = [&](int i) { return (uint32_t)(i / STAGES); };
        auto issue_s = [&](int t, int j) {
            if (j == 0) wait(&q_full[t], 0);
            wait(&kv_full[slot(2 * j)], round(2 * j));
            if (!ok) return;
            tc_fence_after();
            const uint64_t q = dq0 + (uint64_t)((t * Z::Q_BYTES) >> 4);
            const uint64_t k = dk0 + (uint64_t)(slot(2 * j) * (Z::KV_BYTES >> 4));
            const uint32_t d = tmem + t * Z::TILE_COLS + Z::S_COL;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                at_mma(d, q + (((i / 4) * Z::Q_HALF + (i % 4) * 32) >> 4),
                       k + (((i / 4) * Z::KV_HALF + (i % 4) * 32) >> 4), id_s, i > 0 ? 1u : 0u,
                       lead);
            at_commit(&s_full[t], lead);
            __syncwarp();
        };
        for (int t = 0; t < 2; ++t)
            if (ok && (t ? nt1 : nt0) > 0) issue_s(t, 0);
        if (ok) at_commit(&kv_free[slot(0)], lead);
        __syncwarp();
        for (int j = 0; ok && j < n_tiles; ++j) {
            const int vs = slot(2 * j + 1);
            wait(&kv_full[vs], round(2 * j + 1));
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int nt = t ? nt1 : nt0;
                if (!ok || j >= nt) continue;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    wait(&p_full[2 * t + half], (uint32_t)j);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t o = tmem + t * Z::TILE_COLS;
                    const uint64_t v = dv0 + (uint64_t)(vs * (Z::KV_BYTES >> 4));
#pragma unroll
                    for (int part = PARTS - 1; part >= 0; --part)
#pragma unroll
                        for (int i = half * 4; i < half * 4 + 4; ++i)
                            at_mma_tmem_a(o, o + Z::S_COL + part * 64 + i * 8,
                                          v + (uint64_t)((i * 16 * 128) >> 4), id_o,
                                          (j > 0 || i > 0 || part < PARTS - 1) ? 1u : 0u, lead);
                    __syncwarp();
                }
                if (!ok) break;
                if (j + 1 == nt)
                    at_commit(&o_full[t], lead);
                else
                    issue_s(t, j + 1);
            }
            if (!ok) break;
            at_commit(&kv_free[vs], lead);
            if (j + 1 < n_tiles) at_commit(&kv_free[slot(2 * j + 2)], lead);
            __syncwarp();
        }
        // every MMA complete before the tensor memory is released
        at_commit(&fin[0], lead);
        __syncwarp();
        mbar_wait(&fin[0], 0, p.errors);
        __syncwarp();
      } else {
        // ================= K and V, widened =================
        // task k: keys 16 (k % 8) .. + 15 of operand k / 8 (K_0, V_0, K_1, ...)
        const unsigned n_tasks = 16u * n_tiles;
        const int* table = p.block_tables + (size_t)s * p.max_blocks_per_seq;
        // first tile that not every row sees all of
        const unsigned guard_from = (unsigned)max((pos0 + 1) / kMq8Keys - j0, 0);
        // Part i of a task: rows 8 (i / HALVES) + lane / 4, 16 codes from 64 (i %
        // HALVES) + 16 (lane % 4) on.  So eight lanes store to eight bank groups.
        const int r0 = lane / 4, u = lane % 4;
        const size_t row_bytes = (size_t)p.n_kv_heads * D;
        const size_t page_bytes = BS * row_bytes;
        const size_t mine = r0 * row_bytes + (size_t)kvh * D + u * 16;
        const unsigned char* const k_mine = static_cast<const unsigned char*>(p.k_pool) + mine;
        const unsigned char* const v_mine = static_cast<const unsigned char*>(p.v_pool) + mine;
        auto first_key = [&](unsigned k) -> int {
            return (j0 + (int)(k / 16)) * kMq8Keys + (int)(k % 8) * 16;
        };
        // table entry of a task's keys (looked at a task later, when it is there)
        auto entry_of = [&](unsigned k) -> int {
            const int key = first_key(k);
            return k < n_tasks && key < n_keys ? __ldg(table + key / BS) : 0;
        };
        struct Task {
            uint4 codes[kParts];
            float scale;                 // lane 0: of the keys, lane 1: of the values
            bool page;
        };
        auto fetch = [&](Task& t, unsigned k, int entry) {
            const int key0 = first_key(k), left = k < n_tasks ? n_keys - key0 : 0;
            const bool keys = ((k / 8) & 1) == 0;
            t.page = left > 0 && entry >= 0 && entry < p.num_blocks;
            t.scale = 0.f;
            const unsigned char* from = (keys ? k_mine : v_mine) + (size_t)(t.page ? entry : 0) * page_bytes +
                                        (BS > 16 ? (key0 % BS) * row_bytes : 0);
            if (t.page && keys && lane < 2)
                t.scale = __ldg((lane ? p.v_scale : p.k_scale) + (size_t)entry * p.n_kv_heads + kvh);
            if (t.page && left >= 16) {
#pragma unroll
                for (int i = 0; i < kParts; ++i)
                    t.codes[i] = mq8_load(from + i / Z::HALVES * 8 * row_bytes + i % Z::HALVES * 64);
            } else {
                if (!t.page && left > 0) raise_error(p.errors, PKV_DEVERR_BLOCK_ID);
#pragma unroll
                for (int i = 0; i < kParts; ++i)
                    t.codes[i] = t.page && r0 + i / Z::HALVES * 8 < left
                                     ? mq8_load(from + i / Z::HALVES * 8 * row_bytes + i % Z::HALVES * 64)
                                     : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        // where a part's two chunks of 8 go in part 0
        const uint32_t first_at = smem_addr(sKV) + r0 * 128 + (((2 * u) ^ r0) << 4);
        const uint32_t second_at = smem_addr(sKV) + r0 * 128 + (((2 * u + 1) ^ r0) << 4);
        Task now;
        unsigned k = warp - 9;
        fetch(now, k, entry_of(k));
        int entry = entry_of(k + kMq8Widen);
        while (k < n_tasks) {
            const unsigned i_op = k / 8, st = i_op % STAGES, g = k % 8, j = k / 16;
            if (i_op >= STAGES && !__all_sync(0xffffffffu, mbar_wait(&kv_free[st],
                                                                     (i_op / STAGES - 1) & 1u,
                                                                     p.errors)))
                break;
            if ((i_op & 1) == 0) {
                Mq8Scale& e = s_scale[j % kMq8Scales];
                if (lane == 0) {
                    e.a[g] = now.scale;
                } else if (lane == 1) {
                    // (NaN stays)
                    const float b = now.scale < kQ8LeastScale ? kQ8LeastScale : now.scale;
                    const float lb = __log2f(b);
                    e.lb[g] = lb;
                    e.ib[g] = __frcp_rn(b);
                    e.page[g] = now.page ? (mq8_usual(lb) ? 1 : 2) : 0;
                }
            } else if (j >= guard_from) {
                bool any = false;
#pragma unroll
                for (int n = 0; n < kParts; ++n) {
                    uint4& w = now.codes[n];
                    const uint4 bad = make_uint4(q8_nans(w.x), q8_nans(w.y), q8_nans(w.z),
                                                 q8_nans(w.w));
                    any |= (bad.x | bad.y | bad.z | bad.w) != 0u;
                    w = make_uint4(w.x & ~bad.x, w.y & ~bad.y, w.z & ~bad.z, w.w & ~bad.w);
                }
                if (any) *s_poison = 1;
            }
            const uint32_t dst = st * Z::KV_BYTES + g * 2048;
#pragma unroll
            for (int n = 0; n < kParts; ++n) {
                uint4 a, b;
                mq8_widen(now.codes[n], a, b);
                const uint32_t to = dst + n / Z::HALVES * 1024 + n % Z::HALVES * Z::KV_HALF;
                mq8_store(first_at + to, a);
                mq8_store(second_at + to, b);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&kv_full[st]);
            k += kMq8Widen;
            fetch(now, k, entry);
            entry = entry_of(k + kMq8Widen);
        }
      }
    } else {
        // ================= softmax: thread r of group t owns row r of tile t =================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMq8SoftmaxRegs));
        const int t = warp >> 2;
        const int r = (warp & 3) * 32 + lane;
        const int nt = t ? nt1 : nt0;
        if (nt == 0 && cut && t * QT + r / G < rows)
            *reinterpret_cast<float2*>(p.part_ml + 2 * unit_of(t, r)) = make_float2(-INFINITY, 0.f);
        if (nt > 0) {
            const int tok = t * QT + r / G;
            const bool real = tok < rows;
            const int pos = real ? pos0 + tok : -1;        // last key of this row
            const int warp_pos = pos0 + t * QT + ((warp & 3) * 32) / G;
            const size_t row = (size_t)(qs0 + tok_lo + (real ? tok : 0)) * p.n_heads + kvh * G + r % G;
            // ---- the query row, as fp16
            float qf = p.scale_log2;
            {
                const uint4* q4 = reinterpret_cast<const uint4*>(p.q) + row * (D / 8);
                uint4 w[D / 8];
#pragma unroll
                for (int i = 0; i < D / 8; ++i) w[i] = real ? __ldg(q4 + i) : make_uint4(0u, 0u, 0u, 0u);
                if (p.q_bf16) {
                    float top = 0.f;
                    uint32_t* x = reinterpret_cast<uint32_t*>(w);
#pragma unroll
                    for (int i = 0; i < D / 2; ++i) {
                        const float2 f = unpack2<__nv_bfloat16>(x[i]);
                        top = fabsf(f.x) < INFINITY ? fmaxf(top, fabsf(f.x)) : top;
                        top = fabsf(f.y) < INFINITY ? fmaxf(top, fabsf(f.y)) : top;
                    }
                    const int e = min(max((int)(__float_as_uint(top) >> 23), 24), 254);
                    const float to = __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23);
                    qf *= __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
                    for (int i = 0; i < D / 2; ++i) {
                        const float2 f = unpack2<__nv_bfloat16>(x[i]);
                        x[i] = pack2<__half>(f.x * to, f.y * to);
                    }
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    *reinterpret_cast<uint4*>(sQ + t * Z::Q_BYTES + (i / 8) * Z::Q_HALF + r * 128 +
                                              (((i % 8) ^ (r & 7)) << 4)) = w[i];
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[t]);
            }
            const uint32_t t_lane = tmem + t * Z::TILE_COLS + ((uint32_t)((warp & 3) * 32) << 16);
            float m = -INFINITY, lb = 0.f;        // the reference (usual ones: lb 0 unless formed)
            bool odd = false;                     // a row of this warp has one that is not
            // scores formed ahead of the maximum: where their factor is not positive,
            // or a row's are so large that y a + add would lose what matters
            bool formed = !(p.scale_log2 > 0.f);
            float l = 0.f;
            auto group_max = [](const float* v) -> float {
                const float a = max3(max3(v[0], v[1], v[2]), v[3], v[4]);
                const float b = max3(max3(v[5], v[6], v[7]), v[8], v[9]);
                const float c = max3(max3(v[10], v[11], v[12]), v[13], v[14]);
                return max3(max3(a, b, c), v[15], v[15]);
            };
            // The reference to (to, to_lb) where `moved`; what is summed up with it.
            auto move = [&](int j, bool moved, float to, float to_lb) {
                float alpha = 1.f;
                if (moved) {
                    if (m != -INFINITY) {
                        alpha = exp2f((m - to) + (lb - to_lb));
                        l *= exp2f(m - to);
                    }
                    m = to;
                    lb = to_lb;
                }
                odd = __any_sync(0xffffffffu, !mq8_usual(lb));
                if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    // O is at rest: the products up to key tile j - 1 completed before
                    // S_j did
                    const float2 a2 = make_float2(alpha, alpha);
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t ov[32];
                        tc_ld32(t_lane + c0, ov);
                        tc_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            const float2 v = __fmul2_rn(
                                make_float2(__uint_as_float(ov[c]), __uint_as_float(ov[c + 1])), a2);
                            ov[c] = __float_as_uint(v.x);
                            ov[c + 1] = __float_as_uint(v.y);
                        }
                        tc_st32(t_lane + c0, ov);
                    }
                }
            };
            // 2^(y mul1 + add1) of 16 keys as 16-bit pairs from w[..][at] on; their sum.
            auto weights = [](const float* y, float mul1, float add1, uint32_t (&w)[PARTS][16],
                              int at) -> float {
                const float2 mul = make_float2(mul1, mul1), add = make_float2(add1, add1);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 e = __ffma2_rn(make_float2(y[2 * i], y[2 * i + 1]), mul, add);
                    const float2 pv = make_float2(exp2f(e.x), exp2f(e.y));
                    sum = __fadd2_rn(sum, pv);
                    w[0][at + i] = pack2<__half>(pv.x, pv.y);
                    if (PARTS > 1) {
                        const float2 rest = __ffma2_rn(unpack2<__half>(w[0][at + i]),
                                                       make_float2(-1.f, -1.f), pv);
                        w[PARTS - 1][at + i] = pack2<__half>(rest.x, rest.y);
                    }
                }
                return sum.x + sum.y;
            };
            auto stored = [&](int half) {
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * t + half]);
            };
            // 32 keys' weights over the scores just read.
            auto store = [&](uint32_t (&w)[PARTS][16], int part) {
#pragma unroll
                for (int i = 0; i < PARTS; ++i)
                    tc_st16(t_lane + Z::S_COL + i * 64 + part * 16, w[i]);
                if (part & 1) stored(part / 2);
            };
            bool ok = true;
            for (int j = 0; j < nt;) {
                ok = __all_sync(0xffffffffu, mbar_wait(&s_full[t], (uint32_t)j & 1u, p.errors));
                if (!ok) break;
                tc_fence_after();
                const Mq8Scale& sc = s_scale[j % kMq8Scales];
                const int key0 = (j0 + j) * kMq8Keys;
                const uint2 pages = *reinterpret_cast<const uint2*>(sc.page);
                const bool whole = key0 + kMq8Keys - 1 <= warp_pos &&
                                   (pages.x & pages.y) == 0x01010101u;
                if (whole && !formed && !odd) {
                    // ---- the usual tile: this warp's rows see all of it (and lb is 0)
                    float y[kMq8Keys];
                    uint32_t* yr = reinterpret_cast<uint32_t*>(y);
                    tc_ld32(t_lane + Z::S_COL, yr);
                    tc_ld32(t_lane + Z::S_COL + 32, yr + 32);
                    tc_ld32(t_lane + Z::S_COL + 64, yr + 64);
                    tc_ld32(t_lane + Z::S_COL + 96, yr + 96);
                    tc_wait_ld();
                    float z = -INFINITY;                  // largest exponent
#pragma unroll
                    for (int g = 0; g < 8; ++g)
                        z = fmaxf(z, fmaf(group_max(y + 16 * g), sc.a[g] * qf, sc.lb[g]));
                    const bool beyond = z - m > Range::GROW;
                    if (__any_sync(0xffffffffu, beyond)) {
                        if (__any_sync(0xffffffffu, real && beyond && fabsf(z) > 32768.f)) {
                            formed = true;
                            continue;              // this tile once more (S is still there)
                        }
                        move(j, beyond, z, 0.f);
                    }
                    const float base = Range::LIFT - (m == -INFINITY ? 0.f : m);
#pragma unroll
                    for (int part = 0; part < 4; ++part) {
                        uint32_t w[PARTS][16];
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const int gg = part * 2 + g;
                            l = fmaf(weights(y + 16 * gg, sc.a[gg] * qf, base + sc.lb[gg], w, g * 8),
                                     sc.ib[gg], l);
                        }
                        store(w, part);
                    }
                } else {
                    // ---- tiles with hidden keys or missing pages, rows with large scores:
                    // 32 keys at a time, once for the maximum and once for the weights
                    // (rows choose values here, not ways)
                    __syncwarp();
                    const int lim = pos - key0;
                    // group g as this row sees it: the score of a unit of y (never 0,
                    // hidden keys are -inf), 0 for a group with nothing to see
                    auto unit = [&](int g) -> float {
                        const float f = sc.a[g] * qf;
                        return 16 * g <= lim && sc.page[g] ? (fabsf(f) < 1.2e-38f ? 1.2e-38f : f)
                                                           : 0.f;
                    };
                    // 32 keys' scores (formed) or products
                    auto scores = [&](float (&y)[32], int part) {
                        tc_ld32(t_lane + Z::S_COL + part * 32, reinterpret_cast<uint32_t*>(y));
                        tc_wait_ld();
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const float f = unit(part * 2 + g);
#pragma unroll
                            for (int c = 16 * g; c < 16 * g + 16; ++c) {
                                const float x = formed ? y[c] * f : y[c];
                                y[c] = part * 32 + c <= lim && f != 0.f ? x : -INFINITY;
                            }
                        }
                    };
                    bool beyond = false;
                    float top = -INFINITY, top_lb = 0.f;
#pragma unroll 1
                    for (int part = 0; part < 4; ++part) {
                        float y[32];
                        scores(y, part);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const float f = unit(part * 2 + g);
                            const float x = __fmul_rn(group_max(y + 16 * g),
                                                      formed || f == 0.f ? 1.f : f);
                            const float b = f == 0.f ? 0.f : sc.lb[part * 2 + g];
                            beyond |= (x - m) + (b - lb) > Range::GROW;
                            if (top == -INFINITY || (x - top) + (b - top_lb) > 0.f) {
                                top = x;
                                top_lb = b;
                            }
                        }
                    }
                    // scales far apart: L by itself, and m never far below a score
                    const bool apart = odd || ((pages.x | pages.y) & 0x02020202u) != 0u;
                    float high = -INFINITY;
                    if (apart) {
#pragma unroll 1
                        for (int part = 0; part < 4; ++part) {
                            float y[32];
                            scores(y, part);
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                const float f = unit(part * 2 + g);
                                high = fmaxf(high, __fmul_rn(group_max(y + 16 * g),
                                                             formed || f == 0.f ? 1.f : f));
                            }
                        }
                    }
                    const bool moves = beyond || high - m > kMq8Above;
                    if (__any_sync(0xffffffffu, moves)) {
                        if (!formed &&
                            __any_sync(0xffffffffu, real && moves &&
                                                        (fabsf(top) > 32768.f || high > 32768.f))) {
                            formed = true;
                            continue;              // this tile once more (S is still there)
                        }
                        float to = beyond ? top : m, to_lb = beyond ? top_lb : lb;
                        auto join = [&] {
                            if (formed || !mq8_usual(to_lb)) return;
                            to += to_lb;
                            to_lb = 0.f;
                        };
                        join();
                        if (apart) {
                            if (l > 0.f) high = fmaxf(high, m + (__log2f(l) - Range::LIFT));
                            if (high - to > kMq8Above) {
                                to_lb += to - high;
                                to = high;
                                join();
                            }
                        }
                        move(j, moves, to, to_lb);
                    }
                    const float mu = m == -INFINITY ? 0.f : m;
                    if (apart) {
#pragma unroll 1
                        for (int part = 0; part < 4; ++part) {
                            float y[32];
                            scores(y, part);
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                const float f = formed ? 1.f : unit(part * 2 + c / 16);
                                // (hidden ones: -inf, where f may be 0)
                                const float x = y[c] == -INFINITY ? y[c]
                                                : formed          ? y[c] - mu
                                                                  : fmaf(y[c], f, -mu);
                                l += exp2f(x + Range::LIFT);
                            }
                        }
                    }
                    const float base = formed ? Range::LIFT - lb : Range::LIFT - (mu + lb);
                    const float ref = apart ? 0.f : formed ? exp2f(lb) : 1.f;
                    // (the first parts lie where scores were already read, the second
                    // ones wait for the end)
                    uint32_t rest[4][16];
#pragma unroll
                    for (int part = 0; part < 4; ++part) {
                        float y[32];
                        uint32_t w[PARTS][16];
                        scores(y, part);
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const float f = unit(part * 2 + g);
                            if (formed) {
#pragma unroll
                                for (int c = 0; c < 16; ++c) y[16 * g + c] -= mu;   // exact first
                            }
                            const float sum = weights(y + 16 * g, formed || f == 0.f ? 1.f : f,
                                                      f == 0.f ? 0.f : base + sc.lb[part * 2 + g],
                                                      w, g * 8);
                            l = fmaf(sum, f != 0.f ? sc.ib[part * 2 + g] * ref : 0.f, l);
                        }
                        tc_st16(t_lane + Z::S_COL + part * 16, w[0]);
                        if (PARTS > 1)
#pragma unroll
                            for (int c = 0; c < 16; ++c) rest[part][c] = w[PARTS - 1][c];
                    }
                    if (PARTS > 1)
#pragma unroll
                        for (int part = 0; part < 4; ++part)
                            tc_st16(t_lane + Z::S_COL + 64 + part * 16, rest[part]);
                    stored(0);
                    stored(1);
                }
                ++j;
            }
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&o_full[t], 0, p.errors));
            if (ok) {
                tc_fence_after();
                // O 2^lb / l, in two factors: either alone may leave fp32's range
                const float root = exp2f(0.5f * lb), inv = l != 0.f ? __frcp_rn(l) * root : 0.f;
                if (cut && real)
                    *reinterpret_cast<float2*>(p.part_ml + 2 * unit_of(t, r)) =
                        make_float2(m, l * Range::UNLIFT);
                const bool poison = *reinterpret_cast<volatile int*>(s_poison) != 0;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    float o[32];
                    __syncwarp();                  // (rows part ways in what follows)
                    tc_ld32(t_lane + c0, reinterpret_cast<uint32_t*>(o));
                    tc_wait_ld();
                    if (!real) continue;
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = o[c] * inv * root;
                    if (poison) {
                        // NaN that was taken out of V, from the rows that see it
#pragma unroll 1
                        for (int key = max(pos0 / kMq8Keys, j0) * kMq8Keys;
                             key <= min(pos, (j0 + part_tiles) * kMq8Keys - 1); ++key) {
                            const int b = p.block_tables[(size_t)s * p.max_blocks_per_seq + key / BS];
                            if (b < 0 || b >= p.num_blocks) continue;
                            const unsigned char* v =
                                static_cast<const unsigned char*>(p.v_pool) +
                                (((size_t)b * BS + key % BS) * p.n_kv_heads + kvh) * D + c0;
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if ((v[c] & 0x7f) == 0x7f) o[c] = NAN;
                        }
                    }
                    const size_t at = (cut ? unit_of(t, r) : row) * D + c0;
                    if (cut) {
                        float4* o4 = reinterpret_cast<float4*>(p.part_o + at);
#pragma unroll
                        for (int c = 0; c < 32; c += 4)
                            o4[c / 4] = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                    } else if (p.out_dtype == PKV_F32) {
                        float4* o4 = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at);
#pragma unroll
                        for (int c = 0; c < 32; c += 4)
                            o4[c / 4] = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                    } else {
                        uint4* o4 = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + at);
#pragma unroll
                        for (int c = 0; c < 32; c += 8)
                            o4[c / 8] = make_uint4(pack_out(o[c], o[c + 1], p.out_dtype),
                                                   pack_out(o[c + 2], o[c + 3], p.out_dtype),
                                                   pack_out(o[c + 4], o[c + 5], p.out_dtype),
                                                   pack_out(o[c + 6], o[c + 7], p.out_dtype));
                    }
                }
            }
        }
    }

    // ---- tensor memory is released after every thread is done with it
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(512u)
                     : "memory");
}

}  // namespace pkv
