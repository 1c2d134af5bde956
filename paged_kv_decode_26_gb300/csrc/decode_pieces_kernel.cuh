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
// tensor rate.  GB300, 64 contexts of 512-4096 tokens, 32 heads: 357 us of 371
// (the rest: weights and merge), 6.9 TB/s of DRAM; 8 contexts of 8K-32K tokens,
// 32/8 heads: 109 us of 123, 6.0 TB/s.
//
// Split: a stream is HW warps, one per kv head of a group of HW = 8, 4, 2 or
// 1 kv heads (the largest that divides n_kv_heads), so the warps of a stream
// read neighbouring rows of the same blocks at about the same time.  The 16-
// token chunks of all (sequence, head group) pairs form one line, cut into
// runs, one per stream, equal whatever the spread of the lengths (and some
// short ones, see decode_pieces_kernel).  A pair cut by a run boundary is merged
// from its pieces.  Each warp has its own ring of chunks in shared
// memory, filled by TMA (its lane 0 refills a slot as soon as the warp has
// used it), and never waits for another warp.
#pragma once

#include "decode_mma_kernel.cuh"
#include "take_over.cuh"
#include "weight_range.cuh"

namespace pkv {

constexpr int kPieceWarps = 8;
constexpr int kPieceThreads = 32 * kPieceWarps;
constexpr int kPieceTokens = 16;      // tokens per chunk
constexpr int kPieceStages = 3;       // chunks in a warp's ring
constexpr int kPieceGroupsMax = 1024; // group starts kept in shared memory
constexpr int kPieceMinRun = 4;       // chunks a stream takes at least
constexpr int kPieceSoon = 2;         // chunks left to load when the next run is asked for
constexpr int kPieceDealt = 128;      // chunks per stream from which short runs are set apart
constexpr int kPieceRest = 5;         // 1 / this of the units is in short runs
constexpr int kPieceExtra = 6;        // short runs per CTA
constexpr int kPieceShort = 8;        // chunks of a short run at least

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
    int ctas;                  // CTAs that share most of the work
    int extra_ctas;            // and CTAs of short runs
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

__host__ __device__ constexpr size_t decode_pieces_ring_bytes(int D) {
    return (size_t)kPieceWarps * kPieceStages * (2 * kPieceTokens * D * 2);
}

// Length of sequence s, clamped to what the call allows.
__device__ __forceinline__ int piece_length(const PieceParams& p, int s) {
    const int n = p.context_lens[s];
    return n < 0 ? 0 : min(n, p.cap_tokens);
}

// Prefix length of group g (sequences g0 .. g1 - 1), -1 for a group that is not
// well formed (the members then decode their whole contexts).
__device__ __forceinline__ int group_prefix(const PieceParams& p, int g, int g0, int g1) {
    const int pl = p.prefix_lens[g];
    const bool ok = g0 >= 0 && g1 >= g0 && g1 <= p.num_seqs && g1 - g0 <= p.max_group &&
                    pl >= 0 && pl <= p.max_prefix && pl % p.block_size == 0;
    return ok ? pl : -1;
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
    const int pl = max(0, group_prefix(p, lo, gs[lo], gs[lo + 1]));
    return n >= pl && p.max_splits > 0 ? pl : 0;
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

struct NoScores {
    __device__ __forceinline__ void operator()(float, float, float, float) const {}
};

// One 16-token chunk (`valid` of its tokens inside the context, 1..16) of one
// kv head's K and V, swizzled [16 x 128 B] boxes at kbase / vbase, into the
// state of its query heads: mma_heads_chunk with two differences that shorten
// the chain of a chunk (a warp waits for nothing else): the score products
// run in two accumulators, and the state's maximum is a reference that stays
// until a score exceeds its range (weight_range.cuh) -- the common chunk then
// needs one vote instead of the maximum over the lanes, and no rescaling of O.
// PRECISE (fp32 outputs): a chunk's products start from zero and join O by fp32
// additions -- the tensor core drops the bits of a product below those of its
// accumulator, so that O came out 5e-6 short over runs of a thousand tokens.
template <int D, typename T, bool PRECISE, class Scores>
__device__ __forceinline__ void piece_chunk(MmaHeads<D>& st, uint32_t kbase, uint32_t vbase,
                                            int valid, float scale_log2, int lane,
                                            const Scores& scores) {
    constexpr int KSTEPS = D / 16;
    constexpr uint32_t BOX = kPieceTokens * 128;
    constexpr bool THIRD = PRECISE && std::is_same<T, __nv_bfloat16>::value;
    const int gid = lane >> 2, tig = lane & 3;
    const int mat = lane >> 3, mrow = lane & 7;
    // ldmatrix matrices: K (tokens 0-7, c), (0-7, c+1), (8-15, c), (8-15, c+1);
    // V transposed: (tokens 0-7, c), (8-15, c), (0-7, c+1), (8-15, c+1)
    const int k_tok = (mat >> 1) * 8 + mrow, k_dc = mat & 1;
    const int v_tok = (mat & 1) * 8 + mrow, v_dc = mat >> 1;

    // ---- S^T = K Q^T: rows = tokens, columns = query heads
    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KSTEPS; ++ks) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4(kbase + (ks / 4) * BOX + swz(k_tok, (ks % 4) * 2 + k_dc), b0, b1, b2, b3);
        const uint32_t a[4] = {b0, b2, b1, b3};
        mma16816<T>(ks & 1 ? s1 : s0, a, st.qb[ks][0], st.qb[ks][1]);
    }
    // this lane: tokens gid (x0, x1) and gid + 8 (x2, x3) of heads 2 tig, 2 tig + 1
    const bool v0 = gid < valid, v1 = gid + 8 < valid;
    const float x0 = v0 ? __fmul_rn(s0[0] + s1[0], scale_log2) : -INFINITY;
    const float x1 = v0 ? __fmul_rn(s0[1] + s1[1], scale_log2) : -INFINITY;
    const float x2 = v1 ? __fmul_rn(s0[2] + s1[2], scale_log2) : -INFINITY;
    const float x3 = v1 ? __fmul_rn(s0[3] + s1[3], scale_log2) : -INFINITY;
    scores(x0, x1, x2, x3);
    using Range = WeightRange<T>;
    float c0 = fmaxf(x0, x2), c1 = fmaxf(x1, x3);
    if (__any_sync(0xffffffffu, c0 - st.m[0] > Range::GROW || c1 - st.m[1] > Range::GROW)) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            c0 = fmaxf(c0, __shfl_xor_sync(0xffffffffu, c0, off));
            c1 = fmaxf(c1, __shfl_xor_sync(0xffffffffu, c1, off));
        }
        const float m0 = fmaxf(st.m[0], c0), m1 = fmaxf(st.m[1], c1);
        const float al0 = m0 == -INFINITY ? 1.f : exp2f(st.m[0] - m0);
        const float al1 = m1 == -INFINITY ? 1.f : exp2f(st.m[1] - m1);
        st.m[0] = m0;
        st.m[1] = m1;
        st.l[0] *= al0;
        st.l[1] *= al1;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            st.o[j][0] *= al0;
            st.o[j][1] *= al1;
            st.o[j][2] *= al0;
            st.o[j][3] *= al1;
        }
    }
    const float mu0 = st.m[0] == -INFINITY ? 0.f : st.m[0];
    const float mu1 = st.m[1] == -INFINITY ? 0.f : st.m[1];
    // (the difference first: see weight_range.cuh; the factor behind, where it is exact)
    auto weight = [](float x, float mu) { return exp2f(x - mu) * (1.f / Range::UNLIFT); };
    const float p0 = weight(x0, mu0), p1 = weight(x1, mu1);
    const float p2 = weight(x2, mu0), p3 = weight(x3, mu1);
    st.l[0] += p0 + p2;
    st.l[1] += p1 + p3;
    // P in two 16-bit parts (hi = round(p), lo = round(p - hi)), packed by
    // token: (head 2 tig, head 2 tig + 1) of token gid and of token gid + 8;
    // bf16 for an fp32 output the rest too (24 bits)
    const uint32_t hA = pack2<T>(p0, p1), hB = pack2<T>(p2, p3);
    const float2 fA = unpack2<T>(hA), fB = unpack2<T>(hB);
    const uint32_t lA = pack2<T>(p0 - fA.x, p1 - fA.y), lB = pack2<T>(p2 - fB.x, p3 - fB.y);
    // ---- P^T as the B operand: this lane (column = head gid) needs tokens
    // 2 tig, 2 tig + 1 (k 0-7) and 2 tig + 8, 2 tig + 9 (k 8-15), which lanes
    // 4 (2 tig) + gid / 2 and 4 (2 tig + 1) + gid / 2 hold (half gid % 2)
    const int srcA = 4 * (2 * tig) + (gid >> 1), srcB = srcA + 4;
    const uint32_t sel = (gid & 1) ? 0x7632u : 0x5410u;   // the half of this lane's head
    auto from = [](uint32_t x, int src) { return __shfl_sync(0xffffffffu, x, src); };
    const uint32_t hAa = from(hA, srcA), hAb = from(hA, srcB);
    const uint32_t hBa = from(hB, srcA), hBb = from(hB, srcB);
    const uint32_t lAa = from(lA, srcA), lAb = from(lA, srcB);
    const uint32_t lBa = from(lB, srcA), lBb = from(lB, srcB);
    // (keys 2 tig, 2 tig + 1) -> low / high half of one register
    const uint32_t bh0 = __byte_perm(hAa, hAb, sel), bh1 = __byte_perm(hBa, hBb, sel);
    const uint32_t bl0 = __byte_perm(lAa, lAb, sel), bl1 = __byte_perm(lBa, lBb, sel);
    uint32_t bt0 = 0u, bt1 = 0u;
    if (THIRD) {
        const float2 gA = unpack2<T>(lA), gB = unpack2<T>(lB);
        const uint32_t tA = pack2<T>(p0 - fA.x - gA.x, p1 - fA.y - gA.y);
        const uint32_t tB = pack2<T>(p2 - fB.x - gB.x, p3 - fB.y - gB.y);
        bt0 = __byte_perm(from(tA, srcA), from(tA, srcB), sel);
        bt1 = __byte_perm(from(tB, srcA), from(tB, srcB), sel);
    }
    // ---- O^T += V^T P^T; V rows past the context may hold anything (NaN
    // included): P is 0 there, but 0 * NaN is not, so those rows are cleared
    // in the A fragments (tokens 2 tig, 2 tig + 1 in a0/a1, 2 tig + 8, 2 tig +
    // 9 in a2/a3)
    uint32_t vm0 = 0xffffffffu, vm1 = 0xffffffffu;
    if (valid < kPieceTokens) {
        vm0 = (tig * 2 < valid ? 0x0000ffffu : 0u) | (tig * 2 + 1 < valid ? 0xffff0000u : 0u);
        vm1 = (tig * 2 + 8 < valid ? 0x0000ffffu : 0u) | (tig * 2 + 9 < valid ? 0xffff0000u : 0u);
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_trans(vbase + (j / 4) * BOX + swz(v_tok, (j % 4) * 2 + v_dc), b0, b1, b2, b3);
        const uint32_t a[4] = {b0 & vm0, b2 & vm0, b1 & vm1, b3 & vm1};
        if (PRECISE) {
            float o[4] = {0.f, 0.f, 0.f, 0.f};
            if (THIRD) mma16816<T>(o, a, bt0, bt1);
            mma16816<T>(o, a, bl0, bl1);
            mma16816<T>(o, a, bh0, bh1);
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[j][e] += o[e];
        } else {
            mma16816<T>(st.o[j], a, bh0, bh1);
            mma16816<T>(st.o[j], a, bl0, bl1);
        }
    }
}

// Normalised rows of a finished (sequence, kv head) to the output.
template <int D, typename T>
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
        if (gid == 0) *reinterpret_cast<float2*>(p.ws_ml + unit * 2) =
                make_float2(st.m[e], l * WeightRange<T>::UNLIFT);
    }
}

// Where a CTA keeps the piece decode in shared memory.
struct PieceShared {
    unsigned char* ring;       // per warp: kPieceStages x (K, V) chunks
    uint64_t* bars;            // per warp: kPieceStages
    int* cum;                  // [257] chunks before each block of 256 sequences
    int* red;                  // [8]
    int* group_starts;         // [kPieceGroupsMax + 1]
    const int* gs;             // the group starts: there, or in global memory
};

// Bytes beside the ring.
constexpr size_t kPieceControlBytes = (size_t)kPieceWarps * kPieceStages * sizeof(uint64_t) +
                                      (257 + 8 + kPieceGroupsMax + 1) * sizeof(int);

__device__ __forceinline__ PieceShared piece_shared(unsigned char* ring, unsigned char* control) {
    PieceShared sh;
    sh.ring = ring;
    sh.bars = reinterpret_cast<uint64_t*>(control);
    sh.cum = reinterpret_cast<int*>(sh.bars + kPieceWarps * kPieceStages);
    sh.red = sh.cum + 257;
    sh.group_starts = sh.red + 8;
    sh.gs = nullptr;
    return sh;
}

// First chunk, context length and number of chunks of sequence i.
template <bool WEIGHTS>
__device__ __forceinline__ int piece_span(const PieceParams& p, const int* gs, int i, int& first,
                                          int& n) {
    n = piece_length(p, i);
    const int start = WEIGHTS ? 0 : piece_start(p, gs, i, n);
    first = start / kPieceTokens;
    return (n + kPieceTokens - 1) / kPieceTokens - first;
}

// The barrier of the piece decode's 256 threads.
__device__ __forceinline__ void piece_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kPieceThreads) : "memory");
}

// By threads 0 .. 255: barriers, group starts, and the chunks before each
// block of 256 sequences, bad lengths and groups flagged, p.start written.  Returns the
// chunks of all sequences.
template <bool WEIGHTS>
__device__ __forceinline__ int piece_plan(const PieceParams& p, PieceShared& sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.num_seqs;
    if (lane == 0) {
        for (int st = 0; st < kPieceStages; ++st) mbar_init(&sh.bars[warp * kPieceStages + st], 1);
        fence_barrier_init();
    }
    sh.gs = p.group_start;
    if (!WEIGHTS && p.num_groups > 0 && p.num_groups <= kPieceGroupsMax) {
        for (int i = threadIdx.x; i <= p.num_groups; i += kPieceThreads)
            sh.group_starts[i] = p.group_start[i];
        sh.gs = sh.group_starts;
        piece_sync();
    }
    if (!WEIGHTS && blockIdx.x == 0)
        for (int g = threadIdx.x; g < p.num_groups; g += kPieceThreads)
            if (group_prefix(p, g, sh.gs[g], sh.gs[g + 1]) < 0)
                raise_error(p.errors, PKV_DEVERR_CONTEXT);
    const int n_blk = (S + 255) / 256;
    int run = 0;
    for (int b = 0; b < n_blk; ++b) {
        const int i = b * 256 + threadIdx.x;
        int c = 0;
        if (i < S) {
            int first, n;
            c = piece_span<WEIGHTS>(p, sh.gs, i, first, n);
            // (any CTA may be taken over before it starts, so all do this,
            // with the same values)
            const int raw_n = p.context_lens[i];
            if (raw_n < 0 || raw_n > p.cap_tokens) raise_error(p.errors, PKV_DEVERR_CONTEXT);
            if (!WEIGHTS) p.start[i] = first * kPieceTokens;
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) c += __shfl_xor_sync(0xffffffffu, c, off);
        if (lane == 0) sh.red[warp] = c;
        piece_sync();
        if (threadIdx.x == 0) sh.cum[b] = run;
#pragma unroll
        for (int w = 0; w < kPieceWarps; ++w) run += sh.red[w];
        piece_sync();
    }
    if (threadIdx.x == 0) sh.cum[n_blk] = run;
    piece_sync();
    return run;
}

// A chunk's K and V: [head_dim / 64][16 tokens][64 elements] each, by one load
// of each, from rows row .. row + 15 of block b, 64-element columns col, ...
__device__ __forceinline__ void piece_load(uint32_t k, const CUtensorMap* tm_k, uint32_t v,
                                           const CUtensorMap* tm_v, uint32_t bar, uint32_t bytes,
                                           int row, int col, int b, uint64_t policy,
                                           uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %10, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%4], %5;\n\t"
        "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%11, %6, %7, %8}], [%4], %9;\n\t"
        "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%2], [%3, {%11, %6, %7, %8}], [%4], %9;\n\t}" ::"r"(k),
        "l"(reinterpret_cast<uint64_t>(tm_k)), "r"(v), "l"(reinterpret_cast<uint64_t>(tm_v)),
        "r"(bar), "r"(bytes), "r"(row), "r"(col), "r"(b), "l"(policy), "r"(lead), "r"(0)
        : "memory");
}

// How the units (sequence, head group, chunk) are cut into runs, one per
// stream v: the first `first` streams share `share` of them equally (the
// runs of the CTAs that start together), the other `more` the rest.
struct PieceRuns {
    long long total, share;
    int first, more;
    __device__ __forceinline__ long long begin(int v) const {
        return v < first ? share * v / first
                         : share + (more > 0 ? (total - share) * (v - first) / more : 0);
    }
};

__device__ __forceinline__ PieceRuns piece_runs(const PieceParams& p, int chunks) {
    PieceRuns r;
    const int per_cta = kPieceWarps / p.stream_heads;
    r.total = (long long)chunks * (p.n_kv_heads / p.stream_heads);
    r.first = (int)min((long long)p.ctas * per_cta, (r.total + kPieceMinRun - 1) / kPieceMinRun);
    r.share = r.total;
    r.more = 0;
    if (p.extra_ctas > 0 && r.total >= (long long)p.ctas * per_cta * kPieceDealt) {
        r.share = r.total - r.total / kPieceRest;
        r.more = (int)min((long long)p.extra_ctas * per_cta, (r.total - r.share) / kPieceShort);
    }
    return r;
}

// Stream of a CTA's warp, -1 where it has no work.
__device__ __forceinline__ int piece_stream(const PieceParams& p, const PieceRuns& r, int cta,
                                            int warp) {
    const int per_cta = kPieceWarps / p.stream_heads;
    const long long k = (long long)(cta < p.ctas ? cta : cta - p.ctas) * per_cta +
                        warp / p.stream_heads;
    if (cta < p.ctas) return k < r.first ? (int)k : -1;
    return k < r.more ? r.first + (int)k : -1;
}

// A place in the line of units: chunk c of (sequence s, head group hg).
struct PieceCursor {
    int s, hg, c;
    int first, end;      // the pair's chunks
    int n;               // its context length
    int left;            // units to the end of the run
    int v;               // the run's stream
};

// The start of stream v's run, by a whole warp.
template <bool WEIGHTS>
__device__ __forceinline__ PieceCursor piece_locate(const PieceParams& p, const PieceShared& sh,
                                                    const PieceRuns& r, int v, int lane) {
    const long long u0 = r.begin(v);
    const int NHG = p.n_kv_heads / p.stream_heads, S = p.num_seqs, n_blk = (S + 255) / 256;
    PieceCursor k;
    k.v = v;
    k.left = (int)(r.begin(v + 1) - u0);
    const int x = (int)(u0 / NHG);
    int b = 0;
    while (b + 1 < n_blk && sh.cum[b + 1] <= x) ++b;
    int cum = sh.cum[b];
    for (int base = b * 256;; base += 32) {
        const int i = base + lane;
        int f = 0, len = 0;
        const int c = i < S ? piece_span<WEIGHTS>(p, sh.gs, i, f, len) : 0;
        int inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, cum + inc > x);
        if (hit || base + 32 >= S) {
            const int l = hit ? __ffs(hit) - 1 : 31;
            const int nch = __shfl_sync(0xffffffffu, c, l);
            k.s = base + l;
            k.first = __shfl_sync(0xffffffffu, f, l);
            k.end = k.first + nch;
            k.n = __shfl_sync(0xffffffffu, len, l);
            const long long off =
                u0 - (long long)NHG * (cum + __shfl_sync(0xffffffffu, inc, l) - nch);
            k.hg = (int)(off / nch);
            k.c = k.first + (int)(off % nch);
            return k;
        }
        cum += __shfl_sync(0xffffffffu, inc, 31);
    }
}

// The next unit of the run.
template <bool WEIGHTS>
__device__ __forceinline__ void piece_advance(const PieceParams& p, const PieceShared& sh,
                                              PieceCursor& k) {
    --k.left;
    if (++k.c < k.end) return;
    if (++k.hg == p.n_kv_heads / p.stream_heads) {
        k.hg = 0;
        if (k.left > 0) {
            int count;
            while (++k.s < p.num_seqs &&
                   (count = piece_span<WEIGHTS>(p, sh.gs, k.s, k.first, k.n)) == 0) {
            }
            k.end = k.first + count;
        }
    }
    k.c = k.first;
}

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// The runs that a CTA takes after its own.
struct PieceNext {
    uint64_t* soon;        // [1] every warp's loads are near the end of the current run
    uint64_t* full;        // [2] the next run is known
    int* cta;              // [2] the CTA whose run it is, -1: none is left
};

// One warp's work on the CTA's runs: kv head warp % stream_heads of each head
// group.  WEIGHTS: scores go to the workspace and whole (sequence, head)s
// straight to the output; otherwise every piece goes to the workspace, where
// the prefix joins it.  The loads run kPieceStages chunks ahead, over the end
// of a run into the next one.  PRECISE: see piece_chunk.
template <int D, typename T, bool WEIGHTS, bool TAKES, bool PRECISE>
__device__ __forceinline__ void piece_worker(const PieceParams& p, const CUtensorMap& tm_k,
                                             const CUtensorMap& tm_v, const PieceShared& sh,
                                             const PieceRuns& runs, const PieceNext& next) {
    constexpr int HALVES = D / 64;
    constexpr uint32_t HALF = HALVES * kPieceTokens * 128;      // a chunk of K (or V)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int HW = p.stream_heads, hw = warp % HW;
    unsigned char* ring = sh.ring + (size_t)warp * kPieceStages * 2 * HALF;
    uint64_t* full = sh.bars + warp * kPieceStages;
    const int per_block = p.block_size / kPieceTokens;
    const uint64_t policy = l2_policy_evict_first();
    const uint32_t lead = lane == 0 ? 1u : 0u;
    if (lane == 0) {
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }

    PieceCursor ld;              // the next chunk to load
    PieceCursor at;              // the chunk to work on
    bool ahead_run = false;      // the loads are in a run that `at` has not reached
    PieceCursor ahead_start;     // its start
    bool more = true;            // there may be a run after ld's (TAKES)
    int win = -1, bid = -1;      // block ids of the pair's chunks win .. win + 31
    uint32_t bad = 0;            // bit st: the slot's chunk has no valid block
    int cta = blockIdx.x, taken = 0;
    ld.left = 0;

    // Moves ld to the next run that has work, if there is one.
    auto next_run = [&](bool own) {
        while (more) {
            if (!TAKES && !own) more = false;
            if (!more) return;
            if (!own) {
                const int slot = (taken + 1) & 1;
                const bool w = mbar_wait(&next.full[slot], (taken >> 1) & 1, p.errors);
                cta = __all_sync(0xffffffffu, w) ? next.cta[slot] : -1;
                __syncwarp();
                ++taken;
                if (cta < 0) {
                    more = false;
                    return;
                }
            }
            own = false;
            const int v = piece_stream(p, runs, cta, warp);
            if (v >= 0) {
                ld = piece_locate<WEIGHTS>(p, sh, runs, v, lane);
                win = -1;
                if (TAKES && ld.left <= kPieceSoon && lane == 0) mbar_arrive(next.soon);
                return;
            }
            if (TAKES && lane == 0) mbar_arrive(next.soon);
        }
    };
    // Whether the next run is known.
    auto known = [&]() -> bool {
        return __all_sync(0xffffffffu, mbar_test(&next.full[(taken + 1) & 1], (taken >> 1) & 1));
    };
    auto issue = [&](int st) {
        if (win < 0 || ld.c < win || ld.c >= win + 32) {
            win = ld.c;
            const int page = (win + lane) / per_block;
            bid = (win + lane < ld.end && page < p.max_blocks_per_seq)
                      ? p.block_tables[(size_t)ld.s * p.max_blocks_per_seq + page]
                      : -1;
            if (win + lane < ld.end && (bid < 0 || bid >= p.num_blocks)) {
                raise_error(p.errors, PKV_DEVERR_BLOCK_ID);
                bid = -1;
            }
        }
        const int b = __shfl_sync(0xffffffffu, bid, ld.c - win);
        if (b < 0) {
            bad |= 1u << st;
            if (lane == 0) mbar_arrive(&full[st]);
        } else {
            bad &= ~(1u << st);
            // every lane runs the loads with one lane's predicate: a branch
            // around them cost 150 cycles a chunk
            const uint32_t dst = smem_addr(ring) + st * 2 * HALF;
            const int row = (ld.c % per_block) * kPieceTokens;
            const int col = (ld.hg * HW + hw) * HALVES;
            piece_load(dst, &tm_k, dst + HALF, &tm_v, smem_addr(&full[st]), 2 * HALF, row, col, b,
                       policy, lead);
        }
        const int s = ld.s, hg = ld.hg;
        piece_advance<WEIGHTS>(p, sh, ld);
        if (ld.s != s || ld.hg != hg) win = -1;
        if (TAKES && ld.left == kPieceSoon && lane == 0) mbar_arrive(next.soon);
    };

    next_run(true);
    if (ld.left == 0) return;
    if (!TAKES) more = false;
    at = ld;
    MmaHeads<D> state;
    bool fresh = true;                 // the next chunk starts a piece
    bool from_start = false;           // the piece holds the pair's first chunk
    const int gid = lane >> 2, tig = lane & 3;
    int st = 0, put = 0, in_flight = 0;
    uint32_t phase = 0;
    for (;;) {
        // ---- keep the ring full
        while (in_flight < kPieceStages) {
            if (ld.left == 0) {
                // (with chunks in flight the warp works on them until the next
                // run is known)
                if (!TAKES || !more || ahead_run || (in_flight > 0 && !known())) break;
                next_run(false);
                if (!more) break;
                if (at.left == 0) {
                    at = ld;
                } else {
                    ahead_run = true;
                    ahead_start = ld;
                }
            }
            issue(put);
            if (++put == kPieceStages) put = 0;
            ++in_flight;
        }
        if (in_flight == 0) break;
        // ---- one chunk
        const int kvh = at.hg * HW + hw, qh0 = kvh * p.group;
        if (fresh) {
            mma_heads_start<D, T>(state,
                                  reinterpret_cast<const T*>(p.q) +
                                      ((size_t)at.s * p.n_heads + qh0) * D,
                                  p.group, lane);
            from_start = at.c == at.first;
            fresh = false;
        }
        const bool w = mbar_wait(&full[st], phase, p.errors);
        if (!__all_sync(0xffffffffu, w)) {
            // the loads still in flight land before the CTA may exit
            for (; in_flight > 0; --in_flight) {
                mbar_wait(&full[st], phase, p.errors);
                if (++st == kPieceStages) {
                    st = 0;
                    phase ^= 1u;
                }
            }
            break;
        }
        const int valid = min(kPieceTokens, at.n - at.c * kPieceTokens);
        if (!((bad >> st) & 1u)) {
            const uint32_t kbase = smem_addr(ring) + st * 2 * HALF;
            if (WEIGHTS) {
                float* row = p.scores + ((size_t)at.s * p.n_heads + qh0 + 2 * tig) * p.score_stride;
                const StoreScores sink{2 * tig < p.group ? row : nullptr,
                                       2 * tig + 1 < p.group ? row + p.score_stride : nullptr,
                                       at.c * kPieceTokens + gid, at.n};
                piece_chunk<D, T, PRECISE>(state, kbase, kbase + HALF, valid, p.scale_log2, lane,
                                         sink);
            } else {
                piece_chunk<D, T, PRECISE>(state, kbase, kbase + HALF, valid, p.scale_log2, lane,
                                         NoScores());
            }
        } else if (WEIGHTS) {
            // a missing block's tokens weigh nothing
            for (int hh = 0; hh < p.group; ++hh)
                if (lane < valid)
                    p.scores[((size_t)at.s * p.n_heads + qh0 + hh) * p.score_stride +
                             at.c * kPieceTokens + lane] = -INFINITY;
        }
        __syncwarp();
        --in_flight;
        if (++st == kPieceStages) {
            st = 0;
            phase ^= 1u;
        }
        // ---- the piece ends with the pair or with the run
        const bool pair_end = at.c + 1 == at.end;
        if (pair_end || at.left == 1) {
            const size_t pair = (size_t)at.s * p.n_kv_heads + kvh;
            if (WEIGHTS && from_start && pair_end) {
                piece_output<D, T>(state, p, at.s, qh0, lane);
            } else {
                const size_t row = from_start ? (size_t)at.s * p.n_heads + qh0
                                              : (size_t)p.num_seqs * p.n_heads +
                                                    ((size_t)at.v * HW + hw) * p.group;
                mma_heads_partial<D>(state, p.ws_o, p.ws_ml, row, 1, p.group, lane,
                                     WeightRange<T>::UNLIFT);
            }
            if (lane == 0) {
                if (from_start) p.seg_first[pair] = at.v;
                if (pair_end) p.seg_last[pair] = at.v;
            }
            fresh = true;
        }
        if (at.left == 1) {
            if (ahead_run) {
                at = ahead_start;
                ahead_run = false;
            }
            // (no run ahead: the ring is empty, the loads take the next run
            // above, and `at` follows)
            else
                at.left = 0;
        } else {
            piece_advance<WEIGHTS>(p, sh, at);
        }
    }
}

inline size_t decode_pieces_smem_bytes(int D) {
    return 1024 + decode_pieces_ring_bytes(D) + 64 + kPieceControlBytes;
}

// The first `ctas` CTAs have a run of each of their streams, an equal part of
// most of the work.  SMs stream at different rates (GB300, equal parts of a
// whole decode: the first done after 293 us, the last after 375, 331 on
// average), so the rest is in short runs of `extra_ctas` more CTAs: a running
// CTA takes them over one after the other (cluster launch control), its loads
// passing from one run to the next without a break.  Warp 8 asks for the next
// one when every warp's loads are near the end of the current run.
// Without TAKES there are no such runs (and no warp 8): work that a GPU is done
// with in a tenth of a millisecond gains nothing from them -- every run adds a
// piece to merge (8 contexts of 8K-32K tokens, grouped heads: 124 us without,
// 138 us with).
template <int D, typename T, bool WEIGHTS, bool TAKES, bool PRECISE>
__global__ void __launch_bounds__(kPieceThreads + (TAKES ? 32 : 0), 1)
    decode_pieces_kernel(const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ PieceParams p) {
    launch_dependents();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char* sm = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    unsigned char* control = sm + decode_pieces_ring_bytes(D);
    uint4* steal = reinterpret_cast<uint4*>(control);
    uint64_t* steal_bar = reinterpret_cast<uint64_t*>(control + 16);
    PieceNext next;
    next.soon = steal_bar + 1;
    next.full = next.soon + 1;
    next.cta = reinterpret_cast<int*>(next.full + 2);
    PieceShared sh = piece_shared(sm, control + 64);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (TAKES && threadIdx.x == kPieceThreads) {
        mbar_init(steal_bar, 1);
        mbar_init(next.soon, kPieceWarps);
        mbar_init(&next.full[0], 1);
        mbar_init(&next.full[1], 1);
        fence_barrier_init();
    }
    int chunks = 0;
    if (warp < kPieceWarps) chunks = piece_plan<WEIGHTS>(p, sh);
    if (TAKES) __syncthreads();
    if (warp < kPieceWarps) {
        piece_worker<D, T, WEIGHTS, TAKES, PRECISE>(p, tm_k, tm_v, sh, piece_runs(p, chunks), next);
    } else {
        for (int k = 0;; ++k) {
            int cta = -1;
            bool ok = __all_sync(0xffffffffu, mbar_wait(next.soon, k & 1, p.errors));
            if (ok) {
                if (lane == 0) steal_cta(steal, steal_bar);
                ok = __all_sync(0xffffffffu, mbar_wait(steal_bar, k & 1, p.errors));
                if (ok) cta = stolen_cta(steal);
                __syncwarp();
            }
            if (lane == 0) {
                next.cta[(k + 1) & 1] = cta;
                mbar_arrive(&next.full[(k + 1) & 1]);
            }
            if (cta < 0) break;
        }
    }
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

__device__ __forceinline__ PieceSet piece_set(const PieceParams& p, int s, int h, int n,
                                              int start) {
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

// Merged output rows, by a CTA: W of its warps per row take the row's pieces in
// turn, so that many pieces (a long context on many streams) are read at once;
// with few pieces one warp does (W = 1, four rows per CTA).  c, s, h: this
// warp's row (`have`: there is one).  s_o: [kFinishWarps, D].
template <int D, int W>
__device__ __forceinline__ void merge_rows(const PieceParams& p, const PieceSet& c, bool have,
                                           int s, int h, float* s_o) {
    constexpr int V = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int k = c.n_pre + c.first + c.extra;
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
    if (have) {
        const float2 ml = merge_ml(p, c, lane, 32);
        const float inv = ml.y != 0.f ? 1.f / ml.y : 0.f;
#pragma unroll 4
        for (int i = warp % W; i < k; i += W) {
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
    }
    if (W > 1) {
#pragma unroll
        for (int e = 0; e < V; e += 2)
            *reinterpret_cast<float2*>(s_o + warp * D + lane * V + e) = make_float2(o[e], o[e + 1]);
        __syncthreads();
        if (warp % W) return;
#pragma unroll
        for (int w = 1; w < W; ++w)
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const float2 x =
                    *reinterpret_cast<const float2*>(s_o + (warp + w) * D + lane * V + e);
                o[e] += x.x;
                o[e + 1] += x.y;
            }
    }
    if (!have) return;
    const size_t at = ((size_t)s * p.n_heads + h) * D + lane * V;
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

// grid x: rows of a sequence, kFinishWarps / W per CTA; y: sequences.
template <int D, int W>
__global__ void __launch_bounds__(kFinishThreads)
    decode_shared_finish_kernel(const __grid_constant__ PieceParams p) {
    __shared__ __align__(16) float s_o[kFinishWarps * D];
    dependency_wait();
    const int s = blockIdx.y, h = blockIdx.x * (kFinishWarps / W) + (threadIdx.x >> 5) / W;
    const bool have = h < p.n_heads;
    merge_rows<D, W>(p, piece_set(p, s, have ? h : 0, piece_length(p, s), p.start[s]), have, s, h,
                     s_o);
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
        if (c.extra || !c.first) merge_rows<D, kFinishWarps>(p, c, true, s, blockIdx.x, s_mem);
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
