// decode_shared_kernel.cuh -- paged_attn_decode_shared's prefixes: the queries
// of a group's sequences against the keys that they share, on tcgen05
// (attn_tc_kernel.cuh's roles).  The rest of every context runs ahead as pieces
// (decode_pieces_kernel.cuh) and decode_shared_finish_kernel merges the two.
//
// A work item is a split of a prefix x a kv head x a pair of row tiles (256
// rows: members x query heads).  The kernel is bound by the tensor cores where
// a group has many rows, by HBM where it has few.  GB300, a document of 16384
// tokens under 256 sequences, 32 query and 8 kv heads: 87 us by itself (72 with
// weights in one part, of which 20 were its first and last steps), the tensor
// pipe active 48 % of it, on 128 of the SMs, a split per SM; of the whole call's
// 177 us the own tokens take 96 and the merge 8.
#pragma once

#include "attn_tc_precise.cuh"

namespace pkv {

// Candidates (group, kv head, split, pair of row tiles), the row tiles
// fastest (they share the keys): this one may be an item.  (Groups that are not
// well formed have none; piece_plan flags them.)
__device__ __forceinline__ bool attn_prefix_candidate(const AttnParams& a, long long x) {
    const int QT = kAtRows / a.group;
    const int tile = (int)(x % a.tiles);
    x /= a.tiles;
    const int split = (int)(x % a.max_splits);
    x /= a.max_splits;
    const int kvh = (int)(x % a.n_kv_heads), g = (int)(x / a.n_kv_heads);
    const int g0 = a.group_start[g], g1 = a.group_start[g + 1];
    const int pl = a.prefix_lens[g];
    const bool valid = g0 >= 0 && g1 >= g0 && g1 <= a.num_seqs && g1 - g0 <= a.max_group &&
                       pl >= 0 && pl <= a.max_prefix && pl % a.block_size == 0;
    return valid && g0 + tile * a.row_tiles * QT < g1 && (long long)split * a.split_tokens < pl;
}

// The item of a candidate, by a whole warp; false: no member holds the prefix.
__device__ __forceinline__ bool attn_prefix_item(const AttnParams& a, long long x, int lane,
                                                 AttnItem& it) {
    const int QT = kAtRows / a.group;
    const int tile = (int)(x % a.tiles);
    x /= a.tiles;
    const int split = (int)(x % a.max_splits);
    x /= a.max_splits;
    const int kvh = (int)(x % a.n_kv_heads), g = (int)(x / a.n_kv_heads);
    const int g0 = a.group_start[g], g1 = a.group_start[g + 1];
    const int pl = a.prefix_lens[g];
    // the prefix is read through the table of the first member
    // that holds all of it
    int m = -1;
    for (int base = g0; m < 0 && base < g1; base += 32) {
        const int i = base + lane;
        const unsigned has = __ballot_sync(
            0xffffffffu, i < g1 && min(a.context_lens[min(i, g1 - 1)],
                                       a.cap_tokens) >= pl);
        if (has) m = base + __ffs(has) - 1;
    }
    if (m < 0) return false;
    it.done = 0;
    it.kvh = kvh;
    const int NT = a.row_tiles * QT, lo = tile * NT;
    it.row0 = g0 + lo;
    it.rows = min(g1 - g0 - lo, NT);
    it.pos0 = 0;
    it.key_row = m;
    it.key0 = split * a.split_tokens;
    it.n_keys = min(a.split_tokens, pl - it.key0);
    it.split = split;
    it.nt[0] = (it.n_keys + kAtKeys - 1) / kAtKeys;
    it.nt[1] = it.rows > QT ? it.nt[0] : 0;
    const int* row = a.block_tables + (size_t)m * a.max_blocks_per_seq +
                     it.key0 / a.block_size;
    const int pages = (it.n_keys + a.block_size - 1) / a.block_size;
    bool bad = false;
#pragma unroll 4
    for (int k = lane; k < pages; k += 32)
        bad |= (unsigned)row[k] >= (unsigned)a.num_blocks;
    if (__any_sync(0xffffffffu, bad)) {
        if (lane == 0) raise_error(a.errors, PKV_DEVERR_BLOCK_ID);
        it.split = -1 - split;
    }
    return true;
}

// With `dynamic` there is a CTA for every candidate: a running one takes its
// own, then, one after the other, those of CTAs that have not started yet.
// Otherwise CTA c takes candidates c, c + grid, ...
template <int D, typename T, bool PRECISE>
__global__ void __launch_bounds__(kAtThreads, 1)
    attn_prefix_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_o,
                       const __grid_constant__ AttnParams p) {
    launch_dependents();
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    unsigned char* sm = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    unsigned char* control = sm + attn_tile_bytes(D, p.stages);
    uint4* steal = reinterpret_cast<uint4*>(control);
    uint64_t* steal_bar = reinterpret_cast<uint64_t*>(control + 16);
    int* s_tmem = reinterpret_cast<int*>(control + 24);
    AttnControl c = attn_control<D>(sm, control + 32, p.stages);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 8) attn_tmem_alloc(s_tmem);
    if (threadIdx.x == 0) {
        attn_init_barriers(c);
        mbar_init(steal_bar, 1);
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    c.tmem = (uint32_t)*s_tmem;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kAtOtherRegs));
        if (warp == 8) {
            if (PRECISE)
                attn_mma_precise<D, T, true>(c, p, lane);
            else
                attn_mma<D, T, true>(c, p, lane);
        } else if (warp == 9) {
            attn_loader<D, true, PRECISE>(c, p, tm_q, tm_k, tm_v, lane);
        } else if (warp == 11) {
            attn_guard<D, T, true>(c, p, lane);
        } else if (warp == 10) {
            // ---- scheduler; lanes look at 32 candidates at once
            const bool dynamic = p.dynamic != 0;
            const long long stride = dynamic ? p.n_items : gridDim.x;
            uint32_t steal_ph = 0;
            int slot = 0, round = 0;
            bool ok = true;
            auto slot_free = [&]() {
                return round == 0 ||
                       __all_sync(0xffffffffu,
                                  mbar_wait(&c.it_free[slot], (round - 1) & 1, p.errors));
            };
            auto put = [&](const AttnItem& it) {
                if (!(ok = slot_free())) return;
                if (lane == 0) {
                    c.items[slot] = it;
                    mbar_arrive(&c.it_full[slot]);
                }
                if (++slot == kAtItems) {
                    slot = 0;
                    ++round;
                }
            };
            AttnItem it;
            for (long long base = blockIdx.x; ok && base < p.n_items;) {
                const long long i = base + (long long)lane * stride;
                unsigned todo = __ballot_sync(0xffffffffu,
                                              i < p.n_items && attn_prefix_candidate(p, i));
                for (; ok && todo; todo &= todo - 1)
                    if (attn_prefix_item(p, base + (long long)(__ffs(todo) - 1) * stride, lane,
                                         it))
                        put(it);
                base += 32ll * stride;
                if (dynamic && ok) {
                    // ask for another item only when there is a slot for it
                    if (!(ok = slot_free())) break;
                    if (lane == 0) steal_cta(steal, steal_bar);
                    ok = __all_sync(0xffffffffu, mbar_wait(steal_bar, steal_ph, p.errors));
                    steal_ph ^= 1u;
                    if (!ok) break;
                    const int next = stolen_cta(steal);
                    __syncwarp();
                    if (next >= 0) base = next;
                }
            }
            if (ok) {
                it.done = 1;
                put(it);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAtSoftmaxRegs));
        if (!PRECISE)
            attn_softmax<D, T, true>(c, p, tm_o, warp, lane);
        else if (warp < 4)
            attn_softmax_precise<D, T, true>(c, p, warp, lane);
        else
            attn_sum_precise<D, T, true>(c, p, tm_o, warp, lane);
    }

    // ---- tensor memory is released after every thread is done with it
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) attn_tmem_free(c.tmem);
    // the merging kernel waits for this one only: it must not end before the
    // pieces that run ahead of it
    dependency_wait();
}

}  // namespace pkv
