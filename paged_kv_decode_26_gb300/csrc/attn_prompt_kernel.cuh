// attn_prompt_kernel.cuh -- attn_prompt's kernel: causal attention over whole
// packed prompts, by attn_tc_kernel.cuh's roles.
#pragma once

#include "attn_tc_precise.cuh"

namespace pkv {

// The work item i of a launch over whole prompts; false: it is empty.  The
// last tiles of every sequence come first: `band` items of a sequence and kv
// head, then those of the next.
__device__ __forceinline__ bool attn_prompt_item(const AttnParams& p, unsigned i, AttnItem& it) {
    const int G = p.group, QT = kAtRows / G;
    const unsigned band = (unsigned)p.n_kv_heads * p.num_seqs * p.band;
    const unsigned in_band = i % band;
    const int x = (int)(in_band / p.band);
    const int back = (int)(i / band * p.band + in_band % p.band);
    const int s = x / p.n_kv_heads;
    it.done = 0;
    it.kvh = x % p.n_kv_heads;
    const int q0 = p.q_start[s], q1 = p.q_start[s + 1];
    const int len = q1 - q0;
    if (q0 < 0 || len < 0 || q1 > p.total_q || len > p.max_len) {
        if (back == 0 && it.kvh == 0) raise_error(p.errors, PKV_DEVERR_CONTEXT);
        return false;
    }
    const int NT = p.row_tiles * QT;         // tokens per item
    const int lo = ((len + NT - 1) / NT - 1 - back) * NT;
    if (lo < 0 || len == 0) return false;
    it.row0 = q0 + lo;
    it.rows = min(len - lo, NT);
    it.pos0 = lo;
    it.key_row = q0;
    it.key0 = 0;
    it.n_keys = len;
    it.split = 0;
    it.nt[0] = (min(len, lo + QT) + kAtKeys - 1) / kAtKeys;
    it.nt[1] = it.rows > QT ? (min(len, lo + 2 * QT) + kAtKeys - 1) / kAtKeys : 0;
    return true;
}

// Whole prompts.  With `dynamic` there is a CTA for every item: a running one
// takes its own item, then, one after the other, those of CTAs that have not
// started yet.  Otherwise CTA c takes items c, c + grid, ...
template <int D, typename T, bool PRECISE>
__global__ void __launch_bounds__(kAtThreads, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_o,
                       const __grid_constant__ AttnParams p) {
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
                attn_mma_precise<D, T, false>(c, p, lane);
            else
                attn_mma<D, T, false>(c, p, lane);
        } else if (warp == 9) {
            attn_loader<D, false, PRECISE>(c, p, tm_q, tm_k, tm_v, lane);
        } else if (warp == 11) {
            attn_guard<D, T, false>(c, p, lane);
        } else if (warp == 10) {
            // ---- scheduler; lanes look at 32 items at once
            const bool dynamic = p.dynamic != 0;
            const unsigned n_items = (unsigned)p.n_items;
            uint32_t steal_ph = 0;
            int slot = 0, round = 0;
            bool ok = true;
            auto slot_free = [&]() {
                return round == 0 ||
                       __all_sync(0xffffffffu,
                                  mbar_wait(&c.it_free[slot], (round - 1) & 1, p.errors));
            };
            auto put = [&](const AttnItem& it, bool mine) {
                if (mine) {
                    c.items[slot] = it;
                    mbar_arrive(&c.it_full[slot]);
                }
                if (++slot == kAtItems) {
                    slot = 0;
                    ++round;
                }
            };
            for (unsigned base = blockIdx.x; ok;) {
                const unsigned i = base + lane * gridDim.x;
                AttnItem it;
                const bool have = i < n_items && (lane == 0 || !dynamic) &&
                                  attn_prompt_item(p, i, it);
                unsigned todo = __ballot_sync(0xffffffffu, have);
                while (todo && (ok = slot_free())) {
                    put(it, lane == __ffs(todo) - 1);
                    todo &= todo - 1;
                }
                if (!ok) break;
                bool more;
                if (dynamic) {
                    // ask for another item only when there is a slot for it:
                    // what waits here cannot go to an idle SM
                    if (!(ok = slot_free())) break;
                    if (lane == 0) steal_cta(steal, steal_bar);
                    ok = __all_sync(0xffffffffu, mbar_wait(steal_bar, steal_ph, p.errors));
                    steal_ph ^= 1u;
                    if (!ok) break;
                    const int next = stolen_cta(steal);
                    __syncwarp();
                    more = next >= 0;
                    if (more) base = next;
                } else {
                    base += 32 * gridDim.x;
                    more = base < n_items;
                }
                if (!more) {
                    if (slot_free()) {
                        it.done = 1;
                        put(it, lane == 0);
                    }
                    break;
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAtSoftmaxRegs));
        if (!PRECISE)
            attn_softmax<D, T, false>(c, p, tm_o, warp, lane);
        else if (warp < 4)
            attn_softmax_precise<D, T, false>(c, p, warp, lane);
        else
            attn_sum_precise<D, T, false>(c, p, tm_o, warp, lane);
    }

    // ---- tensor memory is released after every thread is done with it
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) attn_tmem_free(c.tmem);
}

}  // namespace pkv
