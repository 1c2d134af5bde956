// decode_pieces_kernel.cuh -- the paged decode as equal pieces per warp, for
// the two decodes that need more than the attention output (sm_103a):
//
//   paged_attn_decode_weights   out, and weights[s, t] += sum_h p[s, h, t]
//   paged_attn_decode_shared    the part of each context behind the prefix
//                               that its group shares (the prefix itself:
//                               attn_tc_kernel.cuh)
//
// Mathematics: scores x_t = scale log2(e) q . K_t, the running maximum M, the
// sum L of 2^(x_t - M) and O = sum 2^(x_t - M) V_t / L per query head; partial
// states merge by the same recurrence.  A token's attention weight is
// 2^(x_t - M) / L with the merged M and L, so it is known only after the last
// piece: the scores go to the workspace (4 bytes per head and token, against
// 4 D bytes of K and V per kv head and token) and a second kernel turns them
// into weights while it merges.
//
// What bounds it: HBM.  Each K and V byte is read once; the products run on
// mma.sync with the tokens as rows (decode_mma_kernel.cuh), far below the
// tensor rate.
//
// Split: a stream is HW warps, one per kv head of a group of HW = 8, 4, 2 or
// 1 kv heads (the largest that divides n_kv_heads), so the warps of a stream
// read neighbouring rows of the same blocks at about the same time.  The 16-
// token chunks of all (sequence, head group) pairs form one line, cut into
// equal runs, one per stream: every warp of the GPU moves the same number of
// bytes whatever the spread of the lengths.  A pair cut by a run boundary is
// merged from its pieces.  Each warp has its own ring of chunks in shared
// memory, filled by TMA (its lane 0 refills a slot as soon as the warp has
// used it), and never waits for another warp.
#pragma once

#include "decode_mma_kernel.cuh"

namespace pkv {

constexpr int kPieceWarps = 8;
constexpr int kPieceThreads = 32 * kPieceWarps;
constexpr int kPieceTokens = 16;      // tokens per chunk
constexpr int kPieceStages = 3;       // chunks in a warp's ring
constexpr int kPieceGroupsMax = 1024; // group starts kept in shared memory

struct PieceParams {
    void* out;
    int out_dtype;
    const void* q;
    const int* block_tables;
    int max_blocks_per_seq;
    const int* context_lens;
    int num_seqs;
    int n_heads;
    int n_kv_heads;
    int group;                 // query heads per kv head
    int block_size;
    int num_blocks;
    int cap_tokens;            // longest context the tables and the caller allow
    float scale_log2;
    int stream_heads;          // kv heads (warps) per stream
    int streams;               // streams of the grid
    int min_run;               // chunks a stream takes at least
    // shared prefixes (group_start NULL: none)
    const int* group_start;    // [num_groups + 1]
    const int* prefix_lens;    // [num_groups]
    int num_groups;
    int max_group;
    int max_prefix;
    int* start;                // [num_seqs]: tokens the prefix kernel covers (written here)
    // prefix partials: row (s * n_heads + h) * max_splits + split
    const float* pre_o;
    const float* pre_ml;
    int split_tokens;
    int max_splits;
    // partial states: rows 0 .. num_seqs * n_heads - 1 for the first piece of
    // a (sequence, head), then stream_heads * group rows per stream for the
    // piece that continues a run
    float* ws_o;               // [rows, D]
    float* ws_ml;              // [rows, 2]
    int* seg_first;            // [num_seqs * n_kv_heads]: stream of the first piece
    int* seg_last;             // and of the last
    float* scores;             // [num_seqs, n_heads, score_stride]
    long long score_stride;
    float* weights;            // [num_seqs, weight_stride]
    long long weight_stride;
    unsigned int* errors;
};

inline size_t decode_pieces_smem_bytes(int D) {
    return 1024 + (size_t)kPieceWarps * kPieceStages * (2 * kPieceTokens * D * 2) +
           (size_t)kPieceWarps * kPieceStages * sizeof(uint64_t) +
           (256 + 8 + kPieceGroupsMax + 2) * sizeof(int);
}

// Length of sequence s, clamped to what the call allows.
__device__ __forceinline__ int piece_length(const PieceParams& p, int s) {
    const int n = p.context_lens[s];
    return n < 0 ? 0 : min(n, p.cap_tokens);
}

// Prefix length of group g, 0 for a group that is not well formed (the
// members then decode their whole contexts).  gs: group starts.
__device__ __forceinline__ int group_prefix(const PieceParams& p, int g, int g0, int g1) {
    const int pl = p.prefix_lens[g];
    const bool ok = g0 >= 0 && g1 >= g0 && g1 <= p.num_seqs && g1 - g0 <= p.max_group &&
                    pl >= 0 && pl <= p.max_prefix && pl % p.block_size == 0;
    return ok ? pl : 0;
}

// Tokens of sequence s (length n) that its group's prefix covers: 0 for a
// sequence in no group or shorter than the prefix.
__device__ __forceinline__ int piece_start(const PieceParams& p, const int* gs, int s, int n) {
    int lo = 0, hi = p.num_groups;          // the last g with gs[g] <= s
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (gs[mid + 1] <= s)
            lo = mid + 1;
        else
            hi = mid;
    }
    if (lo >= p.num_groups || gs[lo] > s) return 0;
    const int pl = group_prefix(p, lo, gs[lo], gs[lo + 1]);
    return n >= pl ? pl : 0;
}

// Writes the scores of one chunk to the workspace: this lane's tokens tok and
// tok + 8 of heads 2 tig and 2 tig + 1.
struct StoreScores {
    float* row0;             // head 2 tig, or NULL past the group
    float* row1;             // head 2 tig + 1
    int tok;
    int n;                   // context length
    __device__ __forceinline__ void operator()(float x0, float x1, float x2, float x3) const {
        if (tok < n) {
            if (row0) row0[tok] = x0;
            if (row1) row1[tok] = x1;
        }
        if (tok + 8 < n) {
            if (row0) row0[tok + 8] = x2;
            if (row1) row1[tok + 8] = x3;
        }
    }
};

// Normalised rows of a finished (sequence, kv head) to the output.
template <int D>
__device__ __forceinline__ void piece_output(const MmaHeads<D>& st, const PieceParams& p, int s,
                                             int qh0, int lane) {
    const int gid = lane >> 2, tig = lane & 3;
    float l0, l1;
    mma_heads_sums<D>(st, l0, l1);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int hh = 2 * tig + e;
        if (hh >= p.group) continue;
        const float l = e ? l1 : l0;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const size_t unit = (size_t)s * p.n_heads + qh0 + hh;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const float a = st.o[j][e] * inv, b = st.o[j][2 + e] * inv;
            const size_t d0 = unit * D + j * 16 + gid, d1 = d0 + 8;
            if (p.out_dtype == PKV_F32) {
                reinterpret_cast<float*>(p.out)[d0] = a;
                reinterpret_cast<float*>(p.out)[d1] = b;
            } else {
                const uint32_t w = pack_out(a, b, p.out_dtype);
                reinterpret_cast<uint16_t*>(p.out)[d0] = (uint16_t)(w & 0xffffu);
                reinterpret_cast<uint16_t*>(p.out)[d1] = (uint16_t)(w >> 16);
            }
        }
        if (gid == 0) *reinterpret_cast<float2*>(p.ws_ml + unit * 2) = make_float2(st.m[e], l);
    }
}

// WEIGHTS: scores go to the workspace and whole (sequence, head)s straight to
// the output; otherwise every piece goes to the workspace, where the prefix
// joins it.
template <int D, typename T, bool WEIGHTS>
__global__ void __launch_bounds__(kPieceThreads, 1)
    decode_pieces_kernel(const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ PieceParams p) {
    constexpr int HALVES = D / 64;
    constexpr uint32_t BOX = kPieceTokens * 128;       // [16 tokens x 64 elements]
    constexpr uint32_t HALF = HALVES * BOX;            // a chunk of K (or V)
    launch_dependents();

    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char* sm = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned char* ring = sm + (size_t)warp * kPieceStages * 2 * HALF;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + (size_t)kPieceWarps * kPieceStages * 2 * HALF);
    uint64_t* full = bars + warp * kPieceStages;
    int* s_cum = reinterpret_cast<int*>(bars + kPieceWarps * kPieceStages);  // [256 + 1]
    int* s_red = s_cum + 257;                                                // [8]
    int* s_gs = s_red + 8;                                                   // group starts

    const int HW = p.stream_heads;
    const int NHG = p.n_kv_heads / HW;
    const int S = p.num_seqs;
    if (lane == 0) {
        for (int st = 0; st < kPieceStages; ++st) mbar_init(&full[st], 1);
        fence_barrier_init();
    }
    const int* gs = p.group_start;
    if (!WEIGHTS && p.num_groups > 0 && p.num_groups <= kPieceGroupsMax) {
        for (int i = threadIdx.x; i <= p.num_groups; i += kPieceThreads) s_gs[i] = p.group_start[i];
        gs = s_gs;
        __syncthreads();
    }

    // first chunk and number of chunks of sequence i
    auto span = [&](int i, int& first, int& n) -> int {
        n = piece_length(p, i);
        const int start = WEIGHTS ? 0 : piece_start(p, gs, i, n);
        first = start / kPieceTokens;
        return (n + kPieceTokens - 1) / kPieceTokens - first;
    };

    // ---- chunks before each block of 256 sequences
    const int n_blk = (S + 255) / 256;
    int run = 0;
    for (int b = 0; b < n_blk; ++b) {
        const int i = b * 256 + threadIdx.x;
        int c = 0;
        if (i < S) {
            int first, n;
            c = span(i, first, n);
            if (blockIdx.x == 0) {
                const int raw_n = p.context_lens[i];
                if (raw_n < 0 || raw_n > p.cap_tokens) raise_error(p.errors, PKV_DEVERR_CONTEXT);
                if (!WEIGHTS) p.start[i] = first * kPieceTokens;
            }
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) c += __shfl_xor_sync(0xffffffffu, c, off);
        if (lane == 0) s_red[warp] = c;
        __syncthreads();
        if (threadIdx.x == 0) s_cum[b] = run;
#pragma unroll
        for (int w = 0; w < kPieceWarps; ++w) run += s_red[w];
        __syncthreads();
    }
    if (threadIdx.x == 0) s_cum[n_blk] = run;
    __syncthreads();

    // ---- this stream's run of units (sequence, head group, chunk)
    const long long total = (long long)run * NHG;
    const long long busy = min((long long)p.streams, (total + p.min_run - 1) / p.min_run);
    const int v = blockIdx.x * (kPieceWarps / HW) + warp / HW;
    if (v < busy) {
        const long long u0 = total * v / busy, u1 = total * (v + 1) / busy;
        const int hw = warp % HW;

        // ---- the sequence of unit u0
        int s = 0, first = 0, n = 0, nch = 0;
        long long off = u0;           // unit's offset within its sequence
        {
            const int x = (int)(u0 / NHG);
            int b = 0;
            while (b + 1 < n_blk && s_cum[b + 1] <= x) ++b;
            int cum = s_cum[b];
            for (int base = b * 256;; base += 32) {
                const int i = base + lane;
                int f = 0, len = 0;
                const int c = i < S ? span(i, f, len) : 0;
                int inc = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, cum + inc > x);
                if (hit || base + 32 >= S) {
                    const int l = hit ? __ffs(hit) - 1 : 31;
                    s = base + l;
                    nch = __shfl_sync(0xffffffffu, c, l);
                    first = __shfl_sync(0xffffffffu, f, l);
                    n = __shfl_sync(0xffffffffu, len, l);
                    off = u0 - (long long)NHG * (cum + __shfl_sync(0xffffffffu, inc, l) - nch);
                    break;
                }
                cum += __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        const int todo = (int)(u1 - u0);
        // consumer: chunk c of (s, hg); producer: the same `stages` ahead
        int hg = (int)(off / nch), c = first + (int)(off % nch);
        int ps = s, phg = hg, pc = c, pfirst = first, pend = first + nch;
        int win = -1, bid = -1;      // block ids of the producer's chunks win .. win + 31
        const int per_block = p.block_size / kPieceTokens;
        uint32_t bad = 0;            // bit st: the slot's chunk has no valid block
        const uint64_t policy = l2_policy_evict_first();
        if (lane == 0) {
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
        }

        auto issue = [&](int st) {
            if (win < 0 || pc < win || pc >= win + 32) {
                win = pc;
                const int page = (win + lane) / per_block;
                bid = (win + lane < pend && page < p.max_blocks_per_seq)
                          ? p.block_tables[(size_t)ps * p.max_blocks_per_seq + page]
                          : -1;
                if (win + lane < pend && (bid < 0 || bid >= p.num_blocks)) {
                    raise_error(p.errors, PKV_DEVERR_BLOCK_ID);
                    bid = -1;
                }
            }
            const int b = __shfl_sync(0xffffffffu, bid, pc - win);
            if (b < 0) {
                bad |= 1u << st;
                if (lane == 0) mbar_arrive(&full[st]);
            } else {
                bad &= ~(1u << st);
                if (lane == 0) {
                    unsigned char* dst = ring + (size_t)st * 2 * HALF;
                    const int row = (pc % per_block) * kPieceTokens;
                    const int col = (phg * HW + hw) * HALVES;
                    mbar_arrive_expect_tx(&full[st], 2 * HALF);
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        tma_load_4d(dst + h * BOX, &tm_k, &full[st], 0, col + h, row, b, policy);
                        tma_load_4d(dst + HALF + h * BOX, &tm_v, &full[st], 0, col + h, row, b,
                                    policy);
                    }
                }
            }
            if (++pc == pend) {
                win = -1;
                if (++phg == NHG) {
                    phg = 0;
                    int len, cnt = 0;
                    while (++ps < S && (cnt = span(ps, pfirst, len)) == 0) {
                    }
                    pend = pfirst + cnt;
                }
                pc = pfirst;
            }
        };

        const int ahead = min(todo, kPieceStages);
        for (int st = 0; st < ahead; ++st) issue(st);

        MmaHeads<D> state;
        bool fresh = true;                 // the next chunk starts a piece
        bool from_start = false;           // the piece holds the pair's first chunk
        int st = 0;
        uint32_t phase = 0;
        const int gid = lane >> 2, tig = lane & 3;
        for (int i = 0; i < todo; ++i) {
            const int kvh = hg * HW + hw, qh0 = kvh * p.group;
            if (fresh) {
                mma_heads_start<D, T>(state,
                                      reinterpret_cast<const T*>(p.q) +
                                          ((size_t)s * p.n_heads + qh0) * D,
                                      p.group, lane);
                from_start = c == first;
                fresh = false;
            }
            const bool w = mbar_wait(&full[st], phase, p.errors);
            if (!__all_sync(0xffffffffu, w)) {
                // the loads still in flight land before the CTA may exit
                for (int j = i; j < todo && j < i + kPieceStages; ++j) {
                    mbar_wait(&full[st], phase, p.errors);
                    if (++st == kPieceStages) {
                        st = 0;
                        phase ^= 1u;
                    }
                }
                break;
            }
            const int valid = min(kPieceTokens, n - c * kPieceTokens);
            if (!((bad >> st) & 1u)) {
                const uint32_t kbase = smem_addr(ring + (size_t)st * 2 * HALF);
                if (WEIGHTS) {
                    float* row = p.scores + ((size_t)s * p.n_heads + qh0 + 2 * tig) * p.score_stride;
                    const StoreScores sink{2 * tig < p.group ? row : nullptr,
                                           2 * tig + 1 < p.group ? row + p.score_stride : nullptr,
                                           c * kPieceTokens + gid, n};
                    mma_heads_chunk<D, T>(state, kbase, kbase + HALF, BOX, 0, valid, p.scale_log2,
                                          lane, sink);
                } else {
                    mma_heads_chunk<D, T>(state, kbase, kbase + HALF, BOX, 0, valid, p.scale_log2,
                                          lane);
                }
            } else if (WEIGHTS) {
                // a missing block's tokens weigh nothing
                for (int hh = 0; hh < p.group; ++hh)
                    if (lane < valid)
                        p.scores[((size_t)s * p.n_heads + qh0 + hh) * p.score_stride +
                                 c * kPieceTokens + lane] = -INFINITY;
            }
            __syncwarp();
            if (i + kPieceStages < todo) issue(st);
            if (++st == kPieceStages) {
                st = 0;
                phase ^= 1u;
            }
            // ---- the piece ends with the pair or with the run
            const bool pair_end = c + 1 == first + nch;
            if (pair_end || i + 1 == todo) {
                const size_t pair = (size_t)s * p.n_kv_heads + kvh;
                if (WEIGHTS && from_start && pair_end) {
                    piece_output<D>(state, p, s, qh0, lane);
                } else {
                    const size_t row = from_start
                                           ? (size_t)s * p.n_heads + qh0
                                           : (size_t)S * p.n_heads + ((size_t)v * HW + hw) * p.group;
                    mma_heads_partial<D>(state, p.ws_o, p.ws_ml, row, 1, p.group, lane);
                }
                if (lane == 0) {
                    if (from_start) p.seg_first[pair] = v;
                    if (pair_end) p.seg_last[pair] = v;
                }
                fresh = true;
            }
            if (pair_end) {
                if (++hg == NHG) {
                    hg = 0;
                    if (i + 1 < todo) {
                        while (++s < S && (nch = span(s, first, n)) == 0) {
                        }
                    }
                }
                c = first;
            } else {
                ++c;
            }
        }
    }
    // the finishing kernel waits for this one only: it must not end before
    // the prefix kernel that runs ahead of it
    if (!WEIGHTS) dependency_wait();
}

// Sum of a (sequence, head)'s partial states: their merged maximum and the
// sum of their weights relative to it.  Pieces: row `row0`, then rows
// slot0 + k * slot_step, k < extra; then n_pre prefix partials from row pre0.
struct PieceSet {
    size_t row0, slot0, slot_step, pre0;
    int first;        // 1: the piece at row0 exists
    int extra;
    int n_pre;
};

__device__ __forceinline__ float2 piece_ml(const PieceParams& p, const PieceSet& c, int i) {
    if (i < c.n_pre) return *reinterpret_cast<const float2*>(p.pre_ml + (c.pre0 + i) * 2);
    i -= c.n_pre;
    const size_t row = i == 0 ? c.row0 : c.slot0 + (size_t)(i - 1) * c.slot_step;
    return *reinterpret_cast<const float2*>(p.ws_ml + row * 2);
}

__device__ __forceinline__ const float* piece_o(const PieceParams& p, const PieceSet& c, int i,
                                                int D) {
    if (i < c.n_pre) return p.pre_o + (c.pre0 + i) * D;
    i -= c.n_pre;
    const size_t row = i == 0 ? c.row0 : c.slot0 + (size_t)(i - 1) * c.slot_step;
    return p.ws_o + row * D;
}

__device__ __forceinline__ PieceSet piece_set(const PieceParams& p, int s, int h, int n, int start) {
    PieceSet c;
    const int kvh = h / p.group;
    const size_t pair = (size_t)s * p.n_kv_heads + kvh;
    c.row0 = (size_t)s * p.n_heads + h;
    c.first = n > start ? 1 : 0;
    const int v0 = c.first ? p.seg_first[pair] : 0, v1 = c.first ? p.seg_last[pair] : 0;
    c.extra = v1 > v0 ? v1 - v0 : 0;
    c.slot_step = (size_t)p.stream_heads * p.group;
    c.slot0 = (size_t)p.num_seqs * p.n_heads + (size_t)(v0 + 1) * c.slot_step +
              (size_t)(kvh % p.stream_heads) * p.group + h % p.group;
    c.n_pre = start > 0 ? (start + p.split_tokens - 1) / p.split_tokens : 0;
    c.pre0 = ((size_t)s * p.n_heads + h) * (size_t)max(p.max_splits, 1);
    return c;
}

// (M, L) of two states joined.
__device__ __forceinline__ float2 join_ml(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x);
    // (an empty state has L = 0; NaN stays NaN)
    const float la = a.y != 0.f ? a.y * exp2f(a.x - m) : 0.f;
    const float lb = b.y != 0.f ? b.y * exp2f(b.x - m) : 0.f;
    return make_float2(m, la + lb);
}

// Merged (M, L) of the pieces, by `lanes` neighbouring lanes of a warp (a
// power of two), lane `sub` of them taking pieces sub, sub + lanes, ...
__device__ __forceinline__ float2 merge_ml(const PieceParams& p, const PieceSet& c, int sub,
                                           int lanes) {
    const int k = c.n_pre + c.first + c.extra;
    float2 ml = make_float2(-INFINITY, 0.f);
#pragma unroll 4
    for (int i = sub; i < k; i += lanes) ml = join_ml(ml, piece_ml(p, c, i));
    for (int off = lanes / 2; off; off >>= 1)
        ml = join_ml(ml, make_float2(__shfl_xor_sync(0xffffffffu, ml.x, off),
                                     __shfl_xor_sync(0xffffffffu, ml.y, off)));
    return ml;
}

constexpr int kFinishThreads = 128;
constexpr int kFinishWarps = kFinishThreads / 32;

// The merged output row of (s, h), by one CTA: its warps take the pieces in
// turn, so that many pieces (a long context on many streams) are read at
// once.  s_o: [kFinishWarps, D].
template <int D>
__device__ __forceinline__ void merge_row(const PieceParams& p, const PieceSet& c, int s, int h,
                                          float* s_o) {
    constexpr int V = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int k = c.n_pre + c.first + c.extra;
    const float2 ml = merge_ml(p, c, lane, 32);
    const float inv = ml.y != 0.f ? 1.f / ml.y : 0.f;
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int i = warp; i < k; i += kFinishWarps) {
        const float2 a = piece_ml(p, c, i);
        const float w = a.y != 0.f ? a.y * exp2f(a.x - ml.x) * inv : 0.f;
        const float* row = piece_o(p, c, i, D) + lane * V;
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 x = *reinterpret_cast<const float2*>(row + e);
            o[e] += w * x.x;
            o[e + 1] += w * x.y;
        }
    }
#pragma unroll
    for (int e = 0; e < V; e += 2)
        *reinterpret_cast<float2*>(s_o + warp * D + lane * V + e) = make_float2(o[e], o[e + 1]);
    __syncthreads();
    const int d = 2 * threadIdx.x;
    if (d >= D) return;
    float2 x = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kFinishWarps; ++w) {
        const float2 y = *reinterpret_cast<const float2*>(s_o + w * D + d);
        x.x += y.x;
        x.y += y.y;
    }
    const size_t at = ((size_t)s * p.n_heads + h) * D + d;
    if (p.out_dtype == PKV_F32)
        *reinterpret_cast<float2*>(reinterpret_cast<float*>(p.out) + at) = x;
    else
        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.out) + at) =
            pack_out(x.x, x.y, p.out_dtype);
}

// One CTA per (head, sequence).
template <int D>
__global__ void __launch_bounds__(kFinishThreads)
    decode_shared_finish_kernel(const __grid_constant__ PieceParams p) {
    __shared__ __align__(16) float s_o[kFinishWarps * D];
    dependency_wait();
    const int s = blockIdx.y, h = blockIdx.x;
    merge_row<D>(p, piece_set(p, s, h, piece_length(p, s), p.start[s]), s, h, s_o);
}

// grid x: n_heads CTAs that merge a head cut into pieces (or empty), then a
// CTA per kWeightTokens tokens that adds their weights; y: sequences.  A
// thread owns four neighbouring tokens and sums their weights over the heads
// in order, so the result does not depend on the launch.
constexpr int kWeightTokens = 4 * kFinishThreads;
template <int D>
__global__ void __launch_bounds__(kFinishThreads)
    decode_weights_finish_kernel(const __grid_constant__ PieceParams p) {
    extern __shared__ __align__(16) float s_mem[];
    dependency_wait();
    const int s = blockIdx.y;
    const int n = piece_length(p, s);
    if ((int)blockIdx.x < p.n_heads) {
        const PieceSet c = piece_set(p, s, blockIdx.x, n, 0);
        if (c.extra || !c.first) merge_row<D>(p, c, s, blockIdx.x, s_mem);
        return;
    }
    const int t0 = (blockIdx.x - p.n_heads) * kWeightTokens;
    if (t0 >= n) return;
    // (M, 1 / L) of every head, four lanes each
    float2* s_ml = reinterpret_cast<float2*>(s_mem);
    for (int h0 = 0; h0 < p.n_heads; h0 += kFinishThreads / 4) {
        const int h = h0 + threadIdx.x / 4;
        PieceSet c = piece_set(p, s, min(h, p.n_heads - 1), n, 0);
        const float2 ml = merge_ml(p, c, threadIdx.x & 3, 4);
        if (h < p.n_heads && (threadIdx.x & 3) == 0)
            s_ml[h] = make_float2(ml.x == -INFINITY ? 0.f : ml.x, ml.y != 0.f ? 1.f / ml.y : 0.f);
    }
    __syncthreads();
    const int t = t0 + 4 * threadIdx.x;
    if (t >= n) return;
    const float* x = p.scores + (size_t)s * p.n_heads * p.score_stride + t;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int h = 0; h < p.n_heads; ++h) {
        const float2 ml = s_ml[h];
        // (rows hold whole chunks of 16: the last ones past the context are
        // read, whatever they hold, and not used)
        const float4 y = __ldcs(reinterpret_cast<const float4*>(x + (size_t)h * p.score_stride));
        w[0] += exp2f(y.x - ml.x) * ml.y;
        w[1] += exp2f(y.y - ml.x) * ml.y;
        w[2] += exp2f(y.z - ml.x) * ml.y;
        w[3] += exp2f(y.w - ml.x) * ml.y;
    }
    float* acc = p.weights + (size_t)s * p.weight_stride + t;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (t + e < n) acc[e] += w[e];
}

}  // namespace pkv
