// evict_kernels.cuh -- a cache cut to a budget by accumulated attention
// weight: kv_evict's two kernels.
//
// Of a sequence of n > keep tokens stay the last `recent` and, of the others,
// the keep - recent with the largest weights (the lower index of equal ones),
// in their order.
//   evict_select_kernel  one CTA per sequence, or a cluster of up to 8 where
//     that leaves SMs idle, finds the smallest weight that stays by three
//     counting passes over the weights' bits (11, 11 and 10 bits, from the
//     top), then lists the tokens that stay in one ordered pass.  It reads 4
//     bytes per token, once: the passes read the keys from shared memory.
//   evict_copy_kernel    moves the listed tokens' K and V rows into the new
//     pages: bound by HBM, each kept row read and written once (GB300, 64
//     sequences cut to 1024 tokens of 8 KB rows: 286 us for both kernels, 6.7
//     TB/s; 4 of 32768 cut to 8192 of 2 KB rows: 60 us, of which the selection,
//     bound by latency, is 21 and the copy of what it lists 35).  A warp takes
//     up to 32 listed tokens, so the page-table lookups of a batch are one
//     coalesced round, and keeps 8 16-byte loads in flight per lane.
// The rows move to other pages, so no copy can overwrite a row that another
// still has to read, and pages that other sequences share stay as they are.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictBins = 2048;
constexpr int kEvictStaged = 48 * 1024;   // keys of a CTA's tokens kept in shared memory
constexpr int kEvictCluster = 8;          // CTAs per sequence at most
// Tokens and columns at most: the passes step by 8192 and round up to 1024 per
// CTA beyond the last one, in 32 bits.
constexpr int kEvictMost = 0x7fffffff - (1 << 14) + 1;

struct EvictParams {
    const int* block_tables;
    int max_blocks_per_seq;
    const int* context_lens;
    const float* weights;
    long long weight_stride;
    int cap_tokens;             // longest context of the tables and the weights' rows
    const int* new_tables;
    int new_blocks_per_seq;
    int* new_lens;
    float* new_weights;
    long long new_weight_stride;
    int new_weight_cols;
    int* kept;                  // [num_seqs, keep]
    int num_seqs;
    int keep;
    int recent;
    int staged;                 // keys that fit the launch's shared memory
    int select_ctas;            // CTAs (a cluster) per sequence
    int block_size;
    int num_blocks;
    uint4* pool[2];
    int row_vec;                // 16-byte vectors per token row
    int parts;                  // column parts per row
    int row_lanes;              // lanes per row: 32, or a power of two that covers a short row
    int batch;                  // kept tokens per unit, at most 32
    unsigned int* errors;
};

// Weights as unsigned numbers of the same order: NaN below everything, the
// two zeros equal.  Bits only (arithmetic would flush small weights to 0).
__device__ __forceinline__ uint32_t weight_key(float w) {
    uint32_t u = __float_as_uint(w);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
    if (u == 0x80000000u) u = 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Length of sequence s, or -1 for one that the call leaves out.
__device__ __forceinline__ int evict_length(const EvictParams& p, int s) {
    const int n = p.context_lens[s];
    return n < 0 || n > p.cap_tokens ? -1 : n;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
            : "memory");
}

// The two ints at `local`'s place in the shared memory of CTA `rank` of the
// cluster (8-byte aligned).
__device__ __forceinline__ int2 cluster_load2(const int* local, int rank) {
    int2 v;
    asm volatile(
        "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\t"
        "ld.shared::cluster.v2.u32 {%0, %1}, [a];\n\t}"
        : "=r"(v.x), "=r"(v.y)
        : "r"(smem_addr(local)), "r"(rank));
    return v;
}

// Sum of the two ints over CTAs 0 .. n - 1 (all loads in flight at once).
__device__ __forceinline__ int2 cluster_sum2(const int* local, int n) {
    int2 v[kEvictCluster], sum = make_int2(0, 0);
#pragma unroll
    for (int r = 0; r < kEvictCluster; ++r)
        v[r] = r < n ? cluster_load2(local, r) : make_int2(0, 0);
#pragma unroll
    for (int r = 0; r < kEvictCluster; ++r) {
        sum.x += v[r].x;
        sum.y += v[r].y;
    }
    return sum;
}

// Sum of x[0 .. warp - 1] for each warp (x: one int per warp, in shared memory).
__device__ __forceinline__ int sum_before(const int* x, int warp, int lane) {
    int v = lane < warp ? x[lane] : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A cluster of `ctas` CTAs per sequence (one where there are enough
// sequences): CTA r owns tokens [r seg, (r + 1) seg) in every pass, and the
// bins and counts of all are added up through distributed shared memory.
__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const EvictParams p) {
    static_assert(kEvictWarps <= 32, "sum_before");
    __shared__ __align__(8) int s_bins[3][kEvictBins];
    __shared__ int s_warp[kEvictWarps], s_warp2[kEvictWarps];
    __shared__ int s_bin, s_above;
    __shared__ __align__(8) int s_cta[2];
    extern __shared__ uint32_t s_keys[];
    launch_dependents();
    const int ctas = p.select_ctas, rank = (int)(blockIdx.x % ctas);
    const int s = blockIdx.x / ctas, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float* w = p.weights + (size_t)s * p.weight_stride;
    int* kept = p.kept + (size_t)s * p.keep;
    float* new_w = p.new_weights + (size_t)s * p.new_weight_stride;
    const int n = evict_length(p, s);
    const int first = rank * kEvictThreads + tid, step = ctas * kEvictThreads;
    if (n <= p.keep) {
        if (n < 0 && first == 0) raise_error(p.errors, PKV_DEVERR_CONTEXT);
        for (int j = first; j < p.keep; j += step) kept[j] = j < n ? j : -1;
        for (int j = first; j < p.new_weight_cols; j += step) new_w[j] = j < n ? w[j] : 0.f;
        if (first == 0) p.new_lens[s] = max(n, 0);
        return;
    }
    for (int j = p.keep + first; j < p.new_weight_cols; j += step) new_w[j] = 0.f;
    if (first == 0) p.new_lens[s] = p.keep;

    const int older = n - p.recent;          // candidates
    int want = p.keep - p.recent;            // of them stay (want < older)
    // this CTA's tokens; warp k owns [k part, (k + 1) part) of them
    const int part = ((n + ctas * kEvictWarps - 1) / (ctas * kEvictWarps) + 31) / 32 * 32;
    const int seg = part * kEvictWarps;
    const int c0 = min(n, rank * seg), c1 = min(n, c0 + seg);
    const int len = max(0, min(older, c1) - c0);       // candidates among them
    // the passes read the keys from shared memory where they fit
    const bool staged = len <= p.staged;
    if (staged) {
#pragma unroll 8
        for (int t = tid; t < len; t += kEvictThreads) s_keys[t] = weight_key(w[c0 + t]);
    }
    for (int b = tid; b < 3 * kEvictBins; b += kEvictThreads) s_bins[0][b] = 0;
    __syncthreads();
    auto key_of = [&](int t) -> uint32_t { return staged ? s_keys[t] : weight_key(w[c0 + t]); };
    // ---- the smallest key that stays, and how many of its equals do
    uint32_t prefix = 0xffffffffu;           // want == 0: no key reaches it
    if (want > 0) {
        uint32_t mask = 0u;
        prefix = 0u;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
            const uint32_t digits = pass == 2 ? 1023u : 2047u;
            int* bins = s_bins[pass];
#pragma unroll 4
            for (int t = tid; t < (len + 31) / 32 * 32; t += kEvictThreads) {
                const uint32_t key = t < len ? key_of(t) : 0u;
                const bool in = t < len && (key & mask) == prefix;
                const int bin = in ? (int)((key >> shift) & digits) : -1;
                // many equal keys in a warp: one addition
                int same;
                __match_all_sync(0xffffffffu, bin, &same);
                if (same) {
                    if (bin >= 0 && lane == 0) atomicAdd(&bins[bin], 32);
                } else if (bin >= 0) {
                    atomicAdd(&bins[bin], 1);
                }
            }
            // the bin that holds the want-th largest: thread i owns the two
            // bins 2 i, 2 i + 1 from the top, of all CTAs
            const int hi = kEvictBins - 1 - 2 * tid;
            int a = 0, b = 0;
            if (ctas > 1) {
                cluster_sync();
                const int2 sum = cluster_sum2(&bins[hi - 1], ctas);
                a = sum.y;
                b = sum.x;
            } else {
                __syncthreads();
                a = bins[hi];
                b = bins[hi - 1];
            }
            int inc = a + b;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (lane == 31) s_warp[warp] = inc;
            __syncthreads();
            const int end = sum_before(s_warp, warp, lane) + inc, start = end - a - b;
            if (start < want && want <= end) {
                const bool top = want <= start + a;
                s_bin = top ? hi : hi - 1;
                s_above = top ? start : start + a;
            }
            __syncthreads();
            want -= s_above;
            prefix |= (uint32_t)s_bin << shift;
            mask |= digits << shift;
        }
    }
    // ---- ordered list
    const int t0 = c0 + warp * part, t1 = min(c1, t0 + part);
    int above = 0, equal = 0;
#pragma unroll 4
    for (int t = t0 + lane; t - lane < t1; t += 32) {
        const uint32_t key = t < t1 && t < older ? key_of(t - c0) : 0u;
        above += __popc(__ballot_sync(0xffffffffu, t < t1 && (t >= older || key > prefix)));
        equal += __popc(__ballot_sync(0xffffffffu, t < t1 && t < older && key == prefix));
    }
    __syncthreads();                         // the last pass's s_warp is read
    if (lane == 0) {
        s_warp[warp] = above;
        s_warp2[warp] = equal;
    }
    __syncthreads();
    int at = sum_before(s_warp, warp, lane), eq = sum_before(s_warp2, warp, lane);
    if (ctas > 1) {
        if (tid == kEvictThreads - 32) {
            s_cta[0] = at + above;
            s_cta[1] = eq + equal;
        }
        cluster_sync();
        const int2 sum = cluster_sum2(s_cta, rank);
        at += sum.x;
        eq += sum.y;
    }
    at += min(eq, want);
    const unsigned below = (1u << lane) - 1u;
#pragma unroll 4
    for (int t = t0 + lane; t - lane < t1; t += 32) {
        const float x = t < t1 ? w[t] : 0.f;
        const uint32_t key = t < t1 && t < older ? key_of(t - c0) : 0u;
        const bool is_eq = t < t1 && t < older && key == prefix;
        const unsigned eq_mask = __ballot_sync(0xffffffffu, is_eq);
        const bool take = (t < t1 && (t >= older || key > prefix)) ||
                          (is_eq && eq + __popc(eq_mask & below) < want);
        const unsigned take_mask = __ballot_sync(0xffffffffu, take);
        if (take) {
            const int j = at + __popc(take_mask & below);
            kept[j] = t;
            new_w[j] = x;
        }
        at += __popc(take_mask);
        eq += __popc(eq_mask);
    }
    if (ctas > 1) cluster_sync();            // others read this CTA's shared memory
}

constexpr int kEvictCopyThreads = 256;
constexpr int kEvictLoads = 8;               // 16-byte loads in flight per lane

// Kept tokens j0 .. j1 - 1 of every sequence.  Units: (sequence, `batch` of
// them, part of the row), the part fastest so that a token's row is read by
// neighbouring warps.  A row's part is taken by LR lanes (32, or fewer for rows
// below 512 bytes: then the warp's lane groups take neighbouring tokens), VEC
// vectors each of K and of V.  RECENT: the last tokens of the context, which
// stay whatever the weights are; otherwise those that the selection lists.
template <int VEC, bool RECENT>
__device__ __forceinline__ void evict_copy(const EvictParams& p, int begin, int end) {
    constexpr int T = kEvictLoads / (2 * VEC);           // tokens per lane group and round
    const int lane = threadIdx.x & 31;
    const int LR = p.row_lanes, groups = 32 / LR;
    const int grp = lane / LR, in_row = lane % LR;
    const int batches = (end - begin + p.batch - 1) / p.batch;
    const long long units = (long long)p.num_seqs * batches * p.parts;
    const long long stride = (long long)gridDim.x * (kEvictCopyThreads / 32);
    for (long long u = (long long)blockIdx.x * (kEvictCopyThreads / 32) + (threadIdx.x >> 5);
         u < units; u += stride) {
        const int part = (int)(u % p.parts);
        const long long sb = u / p.parts;
        const int s = (int)(sb / batches);
        const int j0 = begin + (int)(sb % batches) * p.batch, j = j0 + lane;
        const int n = evict_length(p, s);
        if (n <= p.keep) continue;
        // source and destination row of this lane's token (-1: none)
        long long src = -1, dst = -1;
        if (lane < p.batch && j < end) {
            const int t = RECENT ? n - p.keep + j : p.kept[(size_t)s * p.keep + j];
            const int from = p.block_tables[(size_t)s * p.max_blocks_per_seq + t / p.block_size];
            const int to = p.new_tables[(size_t)s * p.new_blocks_per_seq + j / p.block_size];
            if (from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks) {
                raise_error(p.errors, PKV_DEVERR_BLOCK_ID);
            } else {
                src = ((long long)from * p.block_size + t % p.block_size) * p.row_vec;
                dst = ((long long)to * p.block_size + j % p.block_size) * p.row_vec;
            }
        }
        const int rows = min(p.batch, end - j0);
        const int col = part * (LR * VEC) + in_row;
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += T * groups) {
            uint4 x[T][2][VEC];
            long long to[T];
#pragma unroll
            for (int k = 0; k < T; ++k) {
                const int row = r0 + k * groups + grp;
                const long long a = __shfl_sync(0xffffffffu, src, row & 31);
                const long long b = __shfl_sync(0xffffffffu, dst, row & 31);
                to[k] = row < rows && a >= 0 ? b + col : -1;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int v = 0; v < VEC; ++v)
                        if (to[k] >= 0 && col + v * LR < p.row_vec)
                            x[k][i][v] = __ldcs(p.pool[i] + a + col + v * LR);
            }
#pragma unroll
            for (int k = 0; k < T; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int v = 0; v < VEC; ++v)
                        if (to[k] >= 0 && col + v * LR < p.row_vec)
                            __stcs(p.pool[i] + to[k] + v * LR, x[k][i][v]);
        }
    }
}

// The tokens that stay in any case move while the selection runs.
template <int VEC>
__global__ void __launch_bounds__(kEvictCopyThreads, 3) evict_copy_kernel(const EvictParams p) {
    if (p.recent > 0) evict_copy<VEC, true>(p, p.keep - p.recent, p.keep);
    dependency_wait();
    if (p.keep > p.recent) evict_copy<VEC, false>(p, 0, p.keep - p.recent);
}

}  // namespace pkv
