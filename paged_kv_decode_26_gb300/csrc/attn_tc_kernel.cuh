// attn_tc_kernel.cuh -- attention of many query rows on Blackwell's 5th-
// generation tensor cores (tcgen05), sm_103a, for two operators:
//
//   attn_prompt               whole prompts, packed one after the other, q, k
//                             and v straight from the projections: row i of a
//                             sequence sees its keys t <= i
//   paged_attn_decode_shared  the prefix that a group of sequences shares: the
//                             members' single queries, as the rows of a tile,
//                             see every key of a split of the prefix, read
//                             from its pages once for the whole group; partial
//                             states go to the workspace
//
// Mathematics: S = Q K^T; the running maximum m and sum l of a row; P =
// 2^(a S - m) with a = scale log2(e); O += P V; the result is O / l.
//
// Tiles: 128 rows are 128 / G query tokens (or members) x the G query heads of
// one kv head, so K and V are loaded once for the group.  A CTA works on two
// row tiles at a time (256 rows) that share every K/V tile of 128 keys: while
// the softmax of one tile runs, the tensor core multiplies for the other.
// Products are M = 128, N = 128: 64 cycles of the tensor core for 16 steps of
// the contraction.  Tensor memory holds, per row tile, O (D columns) and S
// (128 columns), which the softmax overwrites with P as 16-bit pairs.
//
// Roles: warps 0-3 and 4-7 are the softmax of tile 0 and 1, a thread per row;
// warp 8 issues every MMA; warp 9 loads by TMA; warp 10 picks the CTA's work
// items; warp 11 guards V tiles that not every row sees all of.  One CTA per SM
// stays for the whole launch: the next item's queries, keys and first products
// overlap the last softmax and the output of the current one.
//
// What bounds it: the tensor core and the softmax in turn.  GB300: two prompts of
// 4096-8192 tokens, 32 heads of 128: 580 us for a call on a cool GPU, 1.60 PFLOP/s
// (0.84 of the burst rate measured for a library product; the tensor pipe is
// active 72 % of the time); 640-650 us when calls follow one another, limited by
// power, 1.44 PFLOP/s (0.76 of that rate, 0.85 of the library's sustained one);
// sixteen of 128-2048 tokens, 32 query and 8 kv heads: 178-185 us, 1.05 PFLOP/s
// (50 %: a sixth of the products are hidden by the causal mask, and eight key
// tiles per item leave its first and last steps in sight).  Pairs of SMs on one
// tile (M = 256) took 1062 us for the first, two threads per softmax row 937.
//
// Precision: S, m, l and O are fp32.  A weight of a prompt is rounded once to the
// 16-bit type of V before the second product (half an eps relative to each
// weight: as much as the rounding of a 16-bit output, and more of it where values
// cancel): the rate of that product rests on it.  A prefix's weights go in two
// parts (attn_weight_parts).  weight_range.cuh keeps fp16 weights clear of its
// smallest numbers; the sum l adds the unrounded weights.  O accumulates in the
// tensor core, which drops what lies below its accumulator's last bit, always
// downwards: up to 2^-23 of O per 16 keys (measured 2e-4 at 32768 keys), so no
// more than the smallest half step of fp16, 2^-12, up to 32768 keys, and of bf16,
// 2^-9, up to 262144.  fp32 outputs are formed otherwise (attn_tc_precise.cuh).
#pragma once

#include "multi_query_tc_kernel.cuh"
#include "take_over.cuh"
#include "weight_range.cuh"

namespace pkv {

constexpr int kAtKeys = 128;        // keys per tile
constexpr int kAtRows = 128;        // rows per row tile
constexpr int kAtThreads = 384;     // 8 softmax warps, MMA, loader, scheduler, guard
// Registers per thread: 384 x 168 at launch = 256 x 200 + 128 x 104 after the
// softmax warps (which hold a row of S) have taken over the others' share.
constexpr int kAtSoftmaxRegs = 200, kAtOtherRegs = 104;
static_assert(256 * kAtSoftmaxRegs + 128 * kAtOtherRegs <= kAtThreads * 168, "registers");
constexpr int kAtItems = 2;         // the item in work and the next one

struct AttnParams {
    void* out;
    int out_dtype;
    int num_seqs;
    int n_heads;
    int n_kv_heads;
    int group;
    float scale_log2;
    int stages;                // slots of the K/V ring
    int row_tiles;             // row tiles per work item: 2, or 1
    int tiles;                 // items of row tiles of the longest sequence / largest group
    int band;                  // prompts: neighbouring items of a sequence and kv head
    long long n_items;
    int dynamic;               // one CTA per item, running CTAs take over waiting ones
    // whole prompts
    const int* q_start;        // [num_seqs + 1]
    int total_q;
    int max_len;
    const void* v;             // token t's row at t * v_stride elements
    long long v_stride;
    // shared prefixes
    const int* group_start;    // [num_groups + 1]
    const int* prefix_lens;    // [num_groups]
    int max_group;
    int max_prefix;
    const int* block_tables;
    int max_blocks_per_seq;
    const int* context_lens;
    int cap_tokens;
    int block_size;
    int num_blocks;
    int split_tokens;          // a multiple of 128
    int max_splits;
    float* pre_o;              // [(seq, head, split), D], normalised
    float* pre_ml;             // [(seq, head, split), 2]
    unsigned int* errors;
};

// One work item: two row tiles of one kv head against n_keys keys.
struct AttnItem {
    int kvh;
    int row0;        // first q token (or member sequence) of tile 0
    int rows;        // tokens left from row0
    int pos0;        // prompt: position of row0 in its sequence
    int key_row;     // prompt: first K/V row; prefix: the sequence whose table is read
    int key0;        // prefix: first key of the split
    int n_keys;      // keys that exist
    int nt[2];       // key tiles per row tile
    int split;       // prefix; negative: -1 - split of an item with a missing page, whose
                     // partial states are empty
    int done;
};

// Sizes in shared and tensor memory.
template <int D>
struct AttnSizes {
    static constexpr int HALVES = D / 64;
    static constexpr uint32_t KV_HALF = kAtKeys * 128;        // [128 keys x 64 elements]
    static constexpr uint32_t KV_BYTES = HALVES * KV_HALF;    // one slot: a K or a V tile
    static constexpr uint32_t Q_HALF = kAtRows * 128;
    static constexpr uint32_t Q_BYTES = HALVES * Q_HALF;
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t TILE_COLS = 256;                // per row tile: O, then S / P
    static constexpr uint32_t S_COL = D;
    static_assert(D % 64 == 0 && D + kAtKeys <= TILE_COLS, "shape");
};
#define PKV_ATTN_SIZES(D)                                                                     \
    [[maybe_unused]] constexpr int HALVES = AttnSizes<D>::HALVES;                             \
    [[maybe_unused]] constexpr uint32_t KV_HALF = AttnSizes<D>::KV_HALF;                      \
    [[maybe_unused]] constexpr uint32_t KV_BYTES = AttnSizes<D>::KV_BYTES;                    \
    [[maybe_unused]] constexpr uint32_t Q_HALF = AttnSizes<D>::Q_HALF;                        \
    [[maybe_unused]] constexpr uint32_t Q_BYTES = AttnSizes<D>::Q_BYTES;                      \
    [[maybe_unused]] constexpr uint32_t TILE_COLS = AttnSizes<D>::TILE_COLS;                  \
    [[maybe_unused]] constexpr uint32_t S_COL = AttnSizes<D>::S_COL;

// 16-bit parts whose sum a softmax weight enters the second product as, for
// 16-bit outputs.  Prefixes: two, the bits of every other decode of these caches
// (a result does not depend on whether a prefix is attended once); one document
// of 16384 tokens under 256 sequences 177 us, 165 with one part, sixteen groups
// 195 and 194; error against 64 bits 1.66e-3 of the outputs' size, that of their
// rounding, and 2.3e-3 with one part.  Prompts: one; two would take packed GQA
// prompts from 183 to 265 us and two of 4096-8192 from 637 to 931, for 1.6e-3
// instead of 2.0e-3.
__host__ __device__ constexpr int attn_weight_parts(bool paged) { return paged ? 2 : 1; }

// Row tiles per work item: fp32 outputs are made one at a time
// (attn_tc_precise.cuh).
__host__ __device__ constexpr int attn_row_tiles(bool precise) { return precise ? 1 : 2; }

// Barriers and item slots of one CTA, behind the tiles in shared memory.
struct AttnControl {
    uint64_t* bars;
    uint64_t* kv_full;      // [stages]
    uint64_t* kv_free;      // [stages]
    uint64_t* land;         // [stages] a V tile for the guard has landed
    uint64_t* q_full;       // [tile]
    uint64_t* q_free;
    uint64_t* s_full;
    uint64_t* p_full;       // [tile][half of the keys]
    uint64_t* o_full;
    uint64_t* o_free;
    uint64_t* it_full;      // [kAtItems]
    uint64_t* it_free;
    uint64_t* fin;
    uint64_t* alpha_full;   // [4]           (attn_tc_precise.cuh)
    uint64_t* row_full;     // [kAtItems]
    AttnItem* items;
    int* poison;            // [kAtItems] V of the item's last tiles held NaN or infinities
    unsigned char* sQ;
    unsigned char* sKV;
    unsigned char* sOut;    // per softmax warp 32 rows x 128 bytes of the output
    uint32_t tmem;
    int stages;
};

__host__ __device__ constexpr int attn_bars(int stages) {
    return 3 * stages + 4 + 2 + 4 + 4 + 2 * kAtItems + 1 + 4 + kAtItems;
}

// Bytes behind the tiles: barriers, item slots, flags.
inline __host__ __device__ size_t attn_control_bytes(int stages) {
    return (size_t)attn_bars(stages) * sizeof(uint64_t) +
           kAtItems * (sizeof(AttnItem) + sizeof(int));
}

template <int D>
__device__ __forceinline__ AttnControl attn_control(unsigned char* tiles, unsigned char* control,
                                                    int stages) {
    AttnControl c;
    c.stages = stages;
    c.sQ = tiles;
    c.sKV = tiles + 2 * AttnSizes<D>::Q_BYTES;
    c.sOut = c.sKV + (size_t)stages * AttnSizes<D>::KV_BYTES;
    c.bars = reinterpret_cast<uint64_t*>(control);
    c.kv_full = c.bars;
    c.kv_free = c.kv_full + stages;
    c.land = c.kv_free + stages;
    c.q_full = c.land + stages;
    c.q_free = c.q_full + 2;
    c.s_full = c.q_free + 2;
    c.p_full = c.s_full + 2;
    c.o_full = c.p_full + 4;
    c.o_free = c.o_full + 2;
    c.it_full = c.o_free + 2;
    c.it_free = c.it_full + kAtItems;
    c.fin = c.it_free + kAtItems;
    c.alpha_full = c.fin + 1;
    c.row_full = c.alpha_full + 4;
    c.items = reinterpret_cast<AttnItem*>(c.row_full + kAtItems);
    c.poison = reinterpret_cast<int*>(c.items + kAtItems);
    c.tmem = 0;
    return c;
}

// By one thread; the CTA's barrier orders it before the first use.
__device__ __forceinline__ void attn_init_barriers(const AttnControl& c) {
    for (int i = 0; i < c.stages; ++i) {
        mbar_init(&c.kv_full[i], 1);
        mbar_init(&c.kv_free[i], 1);
    }
    for (int i = 0; i < c.stages; ++i) mbar_init(&c.land[i], 1);
    for (int t = 0; t < 2; ++t) {
        mbar_init(&c.q_full[t], 1);
        mbar_init(&c.q_free[t], 1);
        mbar_init(&c.s_full[t], 1);
        mbar_init(&c.p_full[2 * t], 4);
        mbar_init(&c.p_full[2 * t + 1], 4);
        mbar_init(&c.o_full[t], 1);
        mbar_init(&c.o_free[t], 4);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&c.alpha_full[i], 4);
    for (int i = 0; i < kAtItems; ++i) {
        mbar_init(&c.it_full[i], 1);
        mbar_init(&c.it_free[i], 11);
        mbar_init(&c.row_full[i], 4);
    }
    mbar_init(c.fin, 1);
    fence_barrier_init();
}

__device__ __forceinline__ void attn_tmem_alloc(int* s_tmem) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(s_tmem)),
                 "r"(AttnSizes<64>::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void attn_tmem_free(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(AttnSizes<64>::TMEM_COLS)
                 : "memory");
}

// Bytes of the queries, the K/V ring and the output rows.
__host__ __device__ constexpr size_t attn_tile_bytes(int D, int stages) {
    return (size_t)2 * kAtRows * D * 2 + (size_t)stages * kAtKeys * D * 2 + 2 * kAtRows * 128;
}

// Dynamic shared memory of attn_prompt_kernel and attn_prefix_kernel.
inline size_t attn_tc_smem_bytes(int D, int stages) {
    return 1024 + attn_tile_bytes(D, stages) + 32 +
           attn_control_bytes(stages);
}

// The largest of three in one instruction (fmaxf's treatment of NaN).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// MMAs issued by the lane with `lead` set; every lane of the warp runs the
// instruction, so descriptors stay in uniform registers.
__device__ __forceinline__ void at_mma(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead));
}
__device__ __forceinline__ void at_mma_tmem_a(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead));
}
__device__ __forceinline__ void at_commit(uint64_t* bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::
            "r"(smem_addr(bar)),
        "r"(lead)
        : "memory");
}

// Whether V of key tile j holds rows that some query row of the item does not
// see (they pass the guard).
template <bool PAGED>
__device__ __forceinline__ bool attn_guarded(const AttnItem& it, int j) {
    return (j + 1) * kAtKeys > (PAGED ? it.n_keys : it.pos0 + 1);
}

// Warp 9: queries, K and V by TMA.  With one row tile per item (PRECISE) items
// take turns with the two places for queries.
template <int D, bool PAGED, bool PRECISE>
__device__ __forceinline__ void attn_loader(const AttnControl& ctl, const AttnParams& p,
                                            const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                            const CUtensorMap& tm_v, int lane) {
    PKV_ATTN_SIZES(D)
    const int G = p.group;
    const int QT = kAtRows / G;
    if (lane == 0) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    const uint64_t keep = l2_policy_evict_normal();   // other row tiles re-read K and V
    const uint64_t once = l2_policy_evict_first();
    int slot = 0, sph = 0;          // item ring
    int st = 0, round = 0;          // K/V ring
    uint32_t q_uses[2] = {0, 0}, n_q = 0;
    bool ok = true;
    const int per_tile = PAGED ? kAtKeys / p.block_size : 0;

    auto next_slot = [&]() {
        if (++st == ctl.stages) {
            st = 0;
            ++round;
        }
    };
    while (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.it_full[slot], sph, p.errors));
        if (!ok) break;
        const AttnItem it = ctl.items[slot];
        if (it.done) break;
        const bool bad = PAGED && it.split < 0;
        const int n_tiles = bad ? 0 : max(it.nt[0], it.nt[1]);
        const int* table = PAGED ? p.block_tables + (size_t)it.key_row * p.max_blocks_per_seq +
                                       it.key0 / p.block_size
                                 : nullptr;
        // pages of key tile j (lane k: page k of the tile)
        auto page_id = [&](int j) -> int {
            const int page = j * per_tile + lane;
            return lane < per_tile && page * p.block_size < it.n_keys ? table[page] : -1;
        };
        int id = PAGED && n_tiles ? page_id(0) : 0;
        for (int j = 0; ok && j < n_tiles; ++j) {
            const int id_next = PAGED && j + 1 < n_tiles ? page_id(j + 1) : 0;
#pragma unroll 1
            for (int kv = 0; ok && kv < 2; ++kv) {
                // K_0, then the queries, then V_0: the order of their use
                if (kv == 1 && j == 0) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (it.nt[t] == 0) continue;
                        const int at = PRECISE ? (int)(n_q & 1) : t;
                        const uint32_t uses = PRECISE ? n_q >> 1 : q_uses[t];
                        if (uses > 0)
                            ok = ok && __all_sync(0xffffffffu, mbar_wait(&ctl.q_free[at],
                                                                         (uses - 1) & 1,
                                                                         p.errors));
                        ++q_uses[t];
                        ++n_q;
                        if (ok && lane == 0) {
                            mbar_arrive_expect_tx(&ctl.q_full[at], Q_BYTES);
#pragma unroll
                            for (int h = 0; h < HALVES; ++h)
                                tma_load_4d(ctl.sQ + at * Q_BYTES + h * Q_HALF, &tm_q,
                                            &ctl.q_full[at], 0, h, it.kvh * G, it.row0 + t * QT,
                                            once);
                        }
                    }
                    if (!ok) break;
                }
                const bool w = round == 0 ||
                               mbar_wait(&ctl.kv_free[st], (round - 1) & 1, p.errors);
                ok = __all_sync(0xffffffffu, w);
                if (!ok) break;
                uint64_t* bar = kv == 1 && attn_guarded<PAGED>(it, j) ? &ctl.land[st]
                                                                      : &ctl.kv_full[st];
                unsigned char* dst = ctl.sKV + (size_t)st * KV_BYTES;
                const CUtensorMap* tm = kv ? &tm_v : &tm_k;
                if (!PAGED) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar, KV_BYTES);
#pragma unroll
                        for (int h = 0; h < HALVES; ++h)
                            tma_load_4d(dst + h * KV_HALF, tm, bar, 0, h, it.kvh,
                                        it.key_row + j * kAtKeys, keep);
                    }
                } else {
                    const unsigned pages = __ballot_sync(0xffffffffu, id >= 0);
                    const uint32_t page_bytes = HALVES * p.block_size * 128;
                    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(pages) * page_bytes);
                    __syncwarp();
                    if (id >= 0) {
#pragma unroll
                        for (int h = 0; h < HALVES; ++h)
                            tma_load_4d(dst + h * KV_HALF + lane * p.block_size * 128, tm, bar,
                                        0, it.kvh * HALVES + h, 0, id, keep);
                    }
                }
                next_slot();
            }
            id = id_next;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.it_free[slot]);
        if (++slot == kAtItems) {
            slot = 0;
            sph ^= 1;
        }
    }
    if (!ok) {
        // a wait gave up: loads in flight get a millisecond to land before the
        // CTA may exit
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
    __syncwarp();
}

// x * 0 + acc of two packed elements.
template <typename T>
__device__ __forceinline__ uint32_t fma2_zero(uint32_t x, uint32_t acc) {
    if (std::is_same<T, __nv_bfloat16>::value)
        asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
    else
        asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
    return acc;
}

// Warp 11: V tiles that hold rows which not every query row sees.  A hidden
// row's weight is 0, but 0 * NaN and 0 * infinity are not, so rows past the
// last key (another sequence's, never loaded, or past the tensor) are cleared,
// and NaN and infinities in rows that only later queries see are taken out
// before the product; the output adds them to the rows that see them.
template <int D, typename T, bool PAGED>
__device__ __forceinline__ void attn_guard(const AttnControl& ctl, const AttnParams& p, int lane) {
    PKV_ATTN_SIZES(D)
    constexpr uint32_t EXP = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
    int slot = 0, sph = 0;          // item ring
    int at = 0;                     // ring slot of the item's K_0
    uint32_t land_ph = 0;           // bit i: phase of land[i] to wait for next
    bool ok = true;
    while (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.it_full[slot], sph, p.errors));
        if (!ok) break;
        const AttnItem it = ctl.items[slot];
        if (it.done) break;
        const int n_tiles = PAGED && it.split < 0 ? 0 : max(it.nt[0], it.nt[1]);
        if (lane == 0) ctl.poison[slot] = 0;
        __syncwarp();
        for (int j = 0; ok && j < n_tiles; ++j) {
            if (!attn_guarded<PAGED>(it, j)) continue;
            const int st = (at + 2 * j + 1) % ctl.stages;
            ok = __all_sync(0xffffffffu, mbar_wait(&ctl.land[st], (land_ph >> st) & 1u, p.errors));
            land_ph ^= 1u << st;
            if (!ok) break;
            unsigned char* v = ctl.sKV + (size_t)st * KV_BYTES;
            const int keys = min(kAtKeys, it.n_keys - j * kAtKeys);
            for (int i = keys * 8 + lane; i < kAtKeys * 8; i += 32)
#pragma unroll
                for (int h = 0; h < HALVES; ++h)
                    *reinterpret_cast<uint4*>(v + h * KV_HALF + i * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
            if (!PAGED) {
                // x * 0 is 0 for every number, NaN for the others: one packed
                // multiply-add per two elements
                uint32_t seen[4] = {0u, 0u, 0u, 0u};
#pragma unroll 8
                for (int i = lane; i < keys * 8; i += 32)
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        const uint4 x =
                            *reinterpret_cast<const uint4*>(v + h * KV_HALF + i * 16);
                        seen[0] = fma2_zero<T>(x.x, seen[0]);
                        seen[1] = fma2_zero<T>(x.y, seen[1]);
                        seen[2] = fma2_zero<T>(x.z, seen[2]);
                        seen[3] = fma2_zero<T>(x.w, seen[3]);
                    }
                const bool bad = ((seen[0] | seen[1] | seen[2] | seen[3]) & 0x7fff7fffu) != 0u;
                if (__any_sync(0xffffffffu, bad)) {
                    if (lane == 0) ctl.poison[slot] = 1;
                    for (int i = lane; i < keys * 64; i += 32)
                        for (int h = 0; h < HALVES; ++h) {
                            uint16_t* e = reinterpret_cast<uint16_t*>(v + h * KV_HALF) + i;
                            if ((*e & EXP) == EXP) *e = 0;
                        }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.kv_full[st]);
        }
        at = (at + 2 * n_tiles) % ctl.stages;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.it_free[slot]);
        if (++slot == kAtItems) {
            slot = 0;
            sph ^= 1;
        }
    }
    __syncwarp();
}

// Warp 8: every MMA.
template <int D, typename T, bool PAGED>
__device__ __forceinline__ void attn_mma(const AttnControl& ctl, const AttnParams& p, int lane) {
    PKV_ATTN_SIZES(D)
    constexpr int PARTS = attn_weight_parts(PAGED);
    const uint32_t id_s = tc_idesc<T>(kAtRows, kAtKeys, 0);
    const uint32_t id_o = tc_idesc<T>(kAtRows, D, 1);
    const uint64_t dq0 = tc_desc_sw128(smem_addr(ctl.sQ), 16, 1024);
    const uint64_t dk0 = tc_desc_sw128(smem_addr(ctl.sKV), 16, 1024);
    const uint64_t dv0 = tc_desc_sw128(smem_addr(ctl.sKV), KV_HALF, 1024);
    const uint32_t lead = elect_one() ? 1u : 0u;
    int slot = 0, sph = 0;
    int st = 0;                         // ring slot of the next tile to use
    uint32_t ph = 0;
    uint32_t n_q[2] = {0, 0}, n_p[2] = {0, 0}, n_o[2] = {0, 0};
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, p.errors));
    };
    // S_t = Q_t K^T with K in slot ks; last: the item's last use of Q_t
    auto issue_s = [&](int t, int ks, bool first, bool last) {
        if (first) {
            wait(&ctl.q_full[t], n_q[t]);
            ++n_q[t];
        }
        if (!ok) return;
        tc_fence_after();
        {
            const uint64_t q = dq0 + (uint64_t)((t * Q_BYTES) >> 4);
            const uint64_t k = dk0 + (uint64_t)(ks * (KV_BYTES >> 4));
            const uint32_t d = ctl.tmem + t * TILE_COLS + S_COL;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                at_mma(d, q + (((i / 4) * Q_HALF + (i % 4) * 32) >> 4),
                       k + (((i / 4) * KV_HALF + (i % 4) * 32) >> 4), id_s, i > 0 ? 1u : 0u, lead);
            at_commit(&ctl.s_full[t], lead);
            if (last) at_commit(&ctl.q_free[t], lead);
        }
        __syncwarp();
    };
    wait(&ctl.it_full[slot], sph);
    AttnItem cur;
    if (ok) cur = ctl.items[slot];
    // ctl.items with a missing page have no products
    auto skip_bad = [&]() {
        while (PAGED && ok && !cur.done && cur.split < 0) {
            if (lane == 0) mbar_arrive(&ctl.it_free[slot]);
            if (++slot == kAtItems) {
                slot = 0;
                sph ^= 1;
            }
            wait(&ctl.it_full[slot], sph);
            if (ok) cur = ctl.items[slot];
        }
    };
    if (ok) skip_bad();
    if (ok && !cur.done) {
        wait(&ctl.kv_full[st], ph);
        for (int t = 0; t < 2; ++t)
            if (ok && cur.nt[t]) issue_s(t, st, true, cur.nt[t] == 1);
        if (ok) at_commit(&ctl.kv_free[st], lead);
        __syncwarp();
        if (++st == ctl.stages) {
            st = 0;
            ph ^= 1u;
        }
    }
    while (ok && !cur.done) {
        const int nt0 = cur.nt[0], nt1 = cur.nt[1];
        const int n_tiles = max(nt0, nt1);
        for (int j = 0; ok && j < n_tiles; ++j) {
            const bool last = j + 1 == n_tiles;
            if (last) {
                // this item's fields are no longer needed; look at the next
                if (lane == 0) mbar_arrive(&ctl.it_free[slot]);
                if (++slot == kAtItems) {
                    slot = 0;
                    sph ^= 1;
                }
                wait(&ctl.it_full[slot], sph);
                if (ok) cur = ctl.items[slot];
                if (ok) skip_bad();
                if (!ok) break;
            }
            const int vs = st;
            wait(&ctl.kv_full[vs], ph);
            if (++st == ctl.stages) {
                st = 0;
                ph ^= 1u;
            }
            const int ks = st;
            const bool have_k = !last || !cur.done;
            bool k_seen = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int nt = t ? nt1 : nt0;
                if (j < nt) {
                    if (j == 0) {
                        if (n_o[t] > 0) wait(&ctl.o_free[t], n_o[t] - 1);
                        ++n_o[t];
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        wait(&ctl.p_full[2 * t + half], n_p[t]);
                        if (!ok) break;
                        tc_fence_after();
                        {
                            const uint32_t o = ctl.tmem + t * TILE_COLS;
                            const uint64_t v = dv0 + (uint64_t)(vs * (KV_BYTES >> 4));
#pragma unroll
                            for (int part = PARTS - 1; part >= 0; --part)
#pragma unroll
                                for (int i = half * 4; i < half * 4 + 4; ++i)
                                    at_mma_tmem_a(o, o + S_COL + part * 64 + i * 8,
                                                  v + (uint64_t)((i * 16 * 128) >> 4), id_o,
                                                  (j > 0 || i > 0 || part < PARTS - 1) ? 1u : 0u,
                                                  lead);
                            if (half && j + 1 == nt) at_commit(&ctl.o_full[t], lead);
                        }
                        __syncwarp();
                    }
                    ++n_p[t];
                }
                if (!ok) break;
                const bool more = last ? !cur.done && cur.nt[t] > 0 : j + 1 < nt;
                if (more) {
                    if (!k_seen) {
                        wait(&ctl.kv_full[ks], ph);
                        k_seen = true;
                    }
                    if (ok)
                        issue_s(t, ks, last, last ? cur.nt[t] == 1 : j + 2 == nt);
                }
            }
            if (!ok) break;
            at_commit(&ctl.kv_free[vs], lead);
            if (have_k) at_commit(&ctl.kv_free[ks], lead);
            __syncwarp();
            if (have_k && ++st == ctl.stages) {
                st = 0;
                ph ^= 1u;
            }
        }
    }
    // every MMA complete before the tensor memory is released
    at_commit(ctl.fin, lead);
    __syncwarp();
    mbar_wait(ctl.fin, 0, p.errors);
    __syncwarp();
}

// 32 rows of 128 bytes (128-byte swizzle) to a box of the output; the warp's
// shared memory may be written again after bulk_read_wait().
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int c1, int c2,
                                             int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];"
        "\n\tcp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(src), "r"(0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void bulk_read_wait() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait() {
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ bool at_finite(float x) { return fabsf(x) <= 3.4e38f; }

// 128 bytes of a thread's output row.  Where the warp's 32 rows all exist they
// go through shared memory and out by TMA in whole lines: a thread's own
// 16-byte stores touch 32 lines an instruction and took a fifth of the time of
// short prompts (GB300, packed prompts of 128-2048 tokens: 185 us, 166 by TMA).
__device__ __forceinline__ void attn_store(const CUtensorMap& tm_o, unsigned char* stage,
                                           unsigned char* own, const uint32_t* w, bool all,
                                           bool real, int c1, int c2, int c3, int lane) {
    if (all) {
        if (lane == 0) bulk_read_wait();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tma_store_4d(&tm_o, smem_addr(stage), c1, c2, c3);
    } else if (real) {
        uint4* o4 = reinterpret_cast<uint4*>(own);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            o4[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
}

// Warps 0-7: thread r of group t owns row r of tile t.
template <int D, typename T, bool PAGED>
__device__ __forceinline__ void attn_softmax(const AttnControl& ctl, const AttnParams& p,
                                             const CUtensorMap& tm_o, int warp, int lane) {
    PKV_ATTN_SIZES(D)
    constexpr int PARTS = attn_weight_parts(PAGED);
    const int G = p.group;
    const int QT = kAtRows / G;
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t t_lane = ctl.tmem + t * TILE_COLS + ((uint32_t)((warp & 3) * 32) << 16);
    const float sc = p.scale_log2;
    int slot = 0, sph = 0;
    uint32_t n_s = 0, n_o = 0;
    bool ok = true;
    while (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.it_full[slot], sph, p.errors));
        if (!ok) break;
        const AttnItem it = ctl.items[slot];
        if (it.done) break;
        const int tok = t * QT + r / G;                // within the item
        const bool real = tok < it.rows;
        const bool bad = PAGED && it.split < 0;
        const int nt = it.nt[t];
        // last key this row sees; rows of no token (never written) may see more
        const int pos = PAGED ? it.n_keys - 1 : it.pos0 + tok;
        const int warp_pos = PAGED ? pos : it.pos0 + t * QT + ((warp & 3) * 32) / G;
        RowReference<T> ref;
        // score = a y; scores formed ahead (a = 1) where the scale is not
        // positive or a row's scores are large (RowReference)
        bool formed = !(sc > 0.f);
        float2 l4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) l4[i] = make_float2(0.f, 0.f);
        if (nt > 0 && !bad) {
            for (int j = 0; j < nt;) {
                ok = __all_sync(0xffffffffu, mbar_wait(&ctl.s_full[t], n_s & 1u, p.errors));
                if (!ok) break;
                tc_fence_after();
                float y[kAtKeys];
                uint32_t* yr = reinterpret_cast<uint32_t*>(y);
                tc_ld32(t_lane + S_COL, yr);
                tc_ld32(t_lane + S_COL + 32, yr + 32);
                tc_ld32(t_lane + S_COL + 64, yr + 64);
                tc_ld32(t_lane + S_COL + 96, yr + 96);
                tc_wait_ld();
                if (formed) {
#pragma unroll
                    for (int c = 0; c < kAtKeys; ++c) y[c] *= sc;
                }
                const float a = formed ? 1.f : sc;
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
                const float x_max = __fmul_rn(mx, a);
                if (__any_sync(0xffffffffu, ref.exceeded(x_max))) {
                    if (!formed && __any_sync(0xffffffffu, real && ref.exceeded(x_max) &&
                                                               ref.beyond(x_max))) {
                        formed = true;
                        continue;                  // this tile once more (S is still there)
                    }
                    const float alpha = ref.take(x_max);
                    if (__any_sync(0xffffffffu, alpha < 1.f)) {
                        // O is at rest: the products up to key tile j - 1
                        // completed before S_j did
                        const float2 a2 = make_float2(alpha, alpha);
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t ov[32];
                            tc_ld32(t_lane + c0, ov);
                            tc_wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; c += 2) {
                                const float2 v = __fmul2_rn(
                                    make_float2(__uint_as_float(ov[c]), __uint_as_float(ov[c + 1])),
                                    a2);
                                ov[c] = __float_as_uint(v.x);
                                ov[c + 1] = __float_as_uint(v.y);
                            }
                            tc_st32(t_lane + c0, ov);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) l4[i] = __fmul2_rn(l4[i], a2);
                    }
                }
                const float2 mul = make_float2(a, a), add = make_float2(ref.add, ref.add);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t w[PARTS][32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int c = half * 64 + 2 * i;
                        const float2 e = __ffma2_rn(make_float2(y[c], y[c + 1]), mul, add);
                        const float2 pv = make_float2(exp2f(e.x), exp2f(e.y));
                        l4[i & 3] = __fadd2_rn(l4[i & 3], pv);
                        w[0][i] = pack2<T>(pv.x, pv.y);
                        if (PARTS > 1) {
                            const float2 rest =
                                __ffma2_rn(unpack2<T>(w[0][i]), make_float2(-1.f, -1.f), pv);
                            w[PARTS - 1][i] = pack2<T>(rest.x, rest.y);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < PARTS; ++k)
                        tc_st32(t_lane + S_COL + k * 64 + half * 32, w[k]);
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.p_full[2 * t + half]);
                }
                ++n_s;
                ++j;
            }
            if (!ok) break;
            ok = __all_sync(0xffffffffu, mbar_wait(&ctl.o_full[t], n_o & 1u, p.errors));
            if (!ok) break;
            ++n_o;
            tc_fence_after();
        }
        if (nt > 0) {
            const float2 la = __fadd2_rn(l4[0], l4[1]), lb = __fadd2_rn(l4[2], l4[3]);
            const float l = (la.x + lb.x) + (la.y + lb.y);
            const float inv = l != 0.f ? 1.f / l : 0.f;
            const int qh = it.kvh * G + r % G;
            const size_t row = (size_t)(it.row0 + tok) * p.n_heads + qh;
            const size_t unit = PAGED ? row * p.max_splits + (bad ? -1 - it.split : it.split)
                                      : row;
            if (PAGED && real)
                *reinterpret_cast<float2*>(p.pre_ml + unit * 2) =
                    make_float2(ref.m, l * ref.unit(ref.m));
            // ---- O / l, 128 bytes of every row at a time (partial states are fp32)
            constexpr int COLS = PAGED ? 32 : 64;
            const int warp_row = (warp & 3) * 32;
            const bool all = t * QT + (warp_row + 31) / G < it.rows;
            const bool poison = !PAGED && ctl.poison[slot] != 0;
            unsigned char* stage = ctl.sOut + warp * 32 * 128;
            unsigned char* own = static_cast<unsigned char*>(PAGED ? p.pre_o : p.out) +
                                 unit * D * (PAGED ? 4 : 2);
#pragma unroll 1
            for (int g = 0; g < D / COLS; ++g) {
                uint32_t w[32];
                __syncwarp();                          // (rows part ways in what follows)
                if (bad) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) w[c] = 0u;
                } else if (PAGED) {
                    tc_ld32(t_lane + g * 32, w);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        w[c] = __float_as_uint(__uint_as_float(w[c]) * inv);
                } else {
                    uint32_t ov[64];
                    tc_ld32(t_lane + g * 64, ov);
                    tc_ld32(t_lane + g * 64 + 32, ov + 32);
                    tc_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        w[c] = pack_out(__uint_as_float(ov[2 * c]) * inv,
                                        __uint_as_float(ov[2 * c + 1]) * inv, p.out_dtype);
                }
                if (poison) {
                    // NaN and infinities that the guard took out of V, from the
                    // rows that this query sees
#pragma unroll 1
                    for (int key = it.pos0 / kAtKeys * kAtKeys; key <= min(pos, it.n_keys - 1);
                         ++key) {
                        const T* v = static_cast<const T*>(p.v) +
                                     (size_t)(it.key_row + key) * p.v_stride + it.kvh * D + g * 64;
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float x = to_float<T>(v[2 * c]), y = to_float<T>(v[2 * c + 1]);
                            if (!at_finite(x) || !at_finite(y)) {
                                const float2 o = p.out_dtype == PKV_BF16
                                                     ? unpack2<__nv_bfloat16>(w[c])
                                                     : unpack2<__half>(w[c]);
                                w[c] = pack_out(at_finite(x) ? o.x : o.x + x,
                                                at_finite(y) ? o.y : o.y + y, p.out_dtype);
                            }
                        }
                    }
                }
                if (!bad && g + 1 == D / COLS) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.o_free[t]);
                }
                attn_store(tm_o, stage, own + g * 128, w, all, real,
                           g + (PAGED ? (bad ? -1 - it.split : it.split) * (D / 32) : 0),
                           it.kvh * G, it.row0 + t * QT + warp_row / G, lane);
            }
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
