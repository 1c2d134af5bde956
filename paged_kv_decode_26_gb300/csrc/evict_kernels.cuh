// evict_kernels.cuh -- a cache cut to a budget by accumulated attention
// weight: kv_evict's two kernels.
//
// Of a sequence of n > keep tokens stay the last `recent` and, of the others,
// the keep - recent with the largest weights (the lower index of equal ones),
// in their order.
//   evict_select_kernel  one CTA per sequence finds the smallest weight that
//     stays by three counting passes over the weights' bits (11, 11 and 10
//     bits, from the top), then lists the tokens that stay in one ordered
//     pass.  It reads 4 bytes per token a pass, from L2 after the first.
//   evict_copy_kernel    moves the listed tokens' K and V rows into the new
//     pages: bound by HBM, each kept row read and written once.  A warp takes
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
constexpr int kEvictStaged = 48 * 1024;   // keys of a sequence kept in shared memory

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
    int block_size;
    int num_blocks;
    uint4* pool[2];
    int row_vec;                // 16-byte vectors per token row
    int parts;                  // column parts per row
    int part_vec;               // vectors per part
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

__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const EvictParams p) {
    __shared__ int s_bins[kEvictBins];
    __shared__ int s_warp[kEvictWarps], s_warp2[kEvictWarps];
    __shared__ int s_bin, s_above;
    launch_dependents();
    const int s = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float* w = p.weights + (size_t)s * p.weight_stride;
    int* kept = p.kept + (size_t)s * p.keep;
    float* new_w = p.new_weights + (size_t)s * p.new_weight_stride;
    const int n = evict_length(p, s);
    if (n < 0 && tid == 0) raise_error(p.errors, PKV_DEVERR_CONTEXT);
    if (n <= p.keep) {
        for (int j = tid; j < p.keep; j += kEvictThreads) kept[j] = j < n ? j : -1;
        for (int j = tid; j < p.new_weight_cols; j += kEvictThreads) new_w[j] = j < n ? w[j] : 0.f;
        if (tid == 0) p.new_lens[s] = max(n, 0);
        return;
    }
    for (int j = p.keep + tid; j < p.new_weight_cols; j += kEvictThreads) new_w[j] = 0.f;
    if (tid == 0) p.new_lens[s] = p.keep;

    const int older = n - p.recent;          // candidates
    int want = p.keep - p.recent;            // of them stay (want < older)
    // the passes below read the keys from shared memory where they fit
    // (a pass over 32768 weights from L2 took 12 us, from there 3)
    extern __shared__ uint32_t s_keys[];
    const bool staged = older <= p.staged;
    if (staged) {
#pragma unroll 8
        for (int t = tid; t < older; t += kEvictThreads) s_keys[t] = weight_key(w[t]);
        __syncthreads();
    }
    auto key_of = [&](int t) -> uint32_t { return staged ? s_keys[t] : weight_key(w[t]); };
    // ---- the smallest key that stays, and how many of its equals do
    uint32_t prefix = 0xffffffffu;           // want == 0: no key reaches it
    if (want > 0) {
        uint32_t mask = 0u;
        prefix = 0u;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
            const uint32_t digits = pass == 2 ? 1023u : 2047u;
            for (int b = tid; b < kEvictBins; b += kEvictThreads) s_bins[b] = 0;
            __syncthreads();
#pragma unroll 4
            for (int t = tid; t < (older + 31) / 32 * 32; t += kEvictThreads) {
                const uint32_t key = t < older ? key_of(t) : 0u;
                const bool in = t < older && (key & mask) == prefix;
                const int bin = in ? (int)((key >> shift) & digits) : -1;
                // many equal keys in a warp: one addition
                int same;
                __match_all_sync(0xffffffffu, bin, &same);
                if (same) {
                    if (bin >= 0 && lane == 0) atomicAdd(&s_bins[bin], 32);
                } else if (bin >= 0) {
                    atomicAdd(&s_bins[bin], 1);
                }
            }
            __syncthreads();
            // the bin that holds the want-th largest: thread i owns the two
            // bins 2 i', 2 i' + 1 from the top
            const int hi = kEvictBins - 1 - 2 * tid;
            const int a = s_bins[hi], b = s_bins[hi - 1];
            int inc = a + b;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (lane == 31) s_warp[warp] = inc;
            __syncthreads();
            int before = 0;
            for (int k = 0; k < warp; ++k) before += s_warp[k];
            const int end = before + inc, start = end - a - b;
            if (start < want && want <= end) {
                const bool first = want <= start + a;
                s_bin = first ? hi : hi - 1;
                s_above = first ? start : start + a;
            }
            __syncthreads();
            want -= s_above;
            prefix |= (uint32_t)s_bin << shift;
            mask |= digits << shift;
            __syncthreads();
        }
    }
    // ---- ordered list: warp k owns tokens [k seg, (k + 1) seg)
    const int seg = ((n + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
    const int t0 = warp * seg, t1 = min(n, t0 + seg);
    int above = 0, equal = 0;
#pragma unroll 4
    for (int t = t0 + lane; t - lane < t1; t += 32) {
        const uint32_t key = t < older ? key_of(t) : 0u;
        above += __popc(__ballot_sync(0xffffffffu, (t < older && key > prefix) ||
                                                       (t >= older && t < n)));
        equal += __popc(__ballot_sync(0xffffffffu, t < older && key == prefix));
    }
    if (lane == 0) {
        s_warp[warp] = above;
        s_warp2[warp] = equal;
    }
    __syncthreads();
    int at = 0, eq = 0;
    for (int k = 0; k < warp; ++k) {
        at += s_warp[k];
        eq += s_warp2[k];
    }
    at += min(eq, want);
    const unsigned below = (1u << lane) - 1u;
#pragma unroll 4
    for (int t = t0 + lane; t - lane < t1; t += 32) {
        const float x = t < n ? w[t] : 0.f;
        const uint32_t key = t < older ? key_of(t) : 0u;
        const bool is_eq = t < older && key == prefix;
        const unsigned eq_mask = __ballot_sync(0xffffffffu, is_eq);
        const bool take = (t < older ? key > prefix : t < n) ||
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
}

constexpr int kEvictCopyThreads = 256;
constexpr int kEvictUnroll = 8;

// Units: (sequence, `batch` kept tokens, pool, part), the part fastest so that a
// token's row is read by neighbouring warps.
__global__ void __launch_bounds__(kEvictCopyThreads) evict_copy_kernel(const EvictParams p) {
    dependency_wait();
    const int lane = threadIdx.x & 31;
    const int batches = (p.keep + p.batch - 1) / p.batch;
    const long long units = (long long)p.num_seqs * batches * 2 * p.parts;
    const long long stride = (long long)gridDim.x * (kEvictCopyThreads / 32);
    for (long long u = (long long)blockIdx.x * (kEvictCopyThreads / 32) + (threadIdx.x >> 5);
         u < units; u += stride) {
        const int part = (int)(u % p.parts);
        const int which = (int)(u / p.parts % 2);
        const long long sb = u / p.parts / 2;
        const int s = (int)(sb / batches), j0 = (int)(sb % batches) * p.batch, j = j0 + lane;
        if (evict_length(p, s) <= p.keep) continue;
        // source and destination row of this lane's token (-1: none)
        long long src = -1, dst = -1;
        if (lane < p.batch && j < p.keep) {
            const int t = p.kept[(size_t)s * p.keep + j];
            const int sb_id = p.block_tables[(size_t)s * p.max_blocks_per_seq + t / p.block_size];
            const int db_id = p.new_tables[(size_t)s * p.new_blocks_per_seq + j / p.block_size];
            if (sb_id < 0 || sb_id >= p.num_blocks || db_id < 0 || db_id >= p.num_blocks) {
                raise_error(p.errors, PKV_DEVERR_BLOCK_ID);
            } else {
                src = ((long long)sb_id * p.block_size + t % p.block_size) * p.row_vec;
                dst = ((long long)db_id * p.block_size + j % p.block_size) * p.row_vec;
            }
        }
        uint4* pool = p.pool[which];
        const int col0 = part * p.part_vec, cols = min(p.part_vec, p.row_vec - col0);
        const int rows = min(p.batch, p.keep - j0);
        // lanes walk the rows x cols vectors of the batch; (row, col) of lane
        int row = lane / cols, col = lane % cols;
        const int dr = 32 / cols, dc = 32 % cols;
        while (__any_sync(0xffffffffu, row < rows)) {
            uint4 r[kEvictUnroll];
            long long to[kEvictUnroll];
#pragma unroll
            for (int k = 0; k < kEvictUnroll; ++k) {
                const long long a = __shfl_sync(0xffffffffu, src, row & 31);
                const long long b = __shfl_sync(0xffffffffu, dst, row & 31);
                to[k] = row < rows && a >= 0 ? b + col0 + col : -1;
                if (to[k] >= 0) r[k] = __ldcs(pool + a + col0 + col);
                row += dr;
                col += dc;
                if (col >= cols) {
                    col -= cols;
                    ++row;
                }
            }
#pragma unroll
            for (int k = 0; k < kEvictUnroll; ++k)
                if (to[k] >= 0) __stcs(pool + to[k], r[k]);
        }
    }
}

}  // namespace pkv
