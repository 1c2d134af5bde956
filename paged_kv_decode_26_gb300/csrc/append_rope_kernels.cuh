// append_rope_kernels.cuh -- new tokens into the paged cache with the rotation
// of their positions on the way: kv_append_rope (16-bit pages) and
// kv_append_rope_q8 (e4m3 pages with a scale per block and kv head), and the
// table of cosines and sines that both read.
//
// Mathematics: a pair (a, b) of a head's elements at angle t becomes
// (a cos t - b sin t, a sin t + b cos t), in fp32, rounded once to what is
// written.  Pair i of rotary_dim / 2 is (i, i + rotary_dim / 2), or the
// neighbours (2 i, 2 i + 1).
//
// What bounds it: HBM, and for a decode step's few tokens the latency of one
// load after the other (slot and position, then table and rows).  So the slot,
// the position and the rows are fetched without waiting for one another, and
// the table's row follows the position.
//
// Split: an item is 16 elements of a head: two 16-byte loads that hold whole
// pairs.  A head is head_dim / 16 items, on neighbouring lanes.  A thread's
// items have the same place in their heads, so the table's row is read once for
// all heads of a token.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

constexpr int kRopeThreads = 256;

struct RopeSource {
    const void* p;          // token t's row at p + t * stride elements
    long long stride;
};

struct AppendRopeParams {
    RopeSource q, k, v;     // q.p NULL: no queries
    void* q_out;            // (NULL: none)
    long long q_out_stride;
    void* k_out;            // the rotated keys, packed (NULL: none)
    long long k_out_stride;
    void* k_pool;
    void* v_pool;
    float* k_scale;         // 8-bit pages: [num_blocks, n_kv_heads]
    float* v_scale;
    const float* table;     // [positions, rotary_dim]: cosines, then sines; NULL: no rotation
    int table_rows;
    int rotary_dim;         // a multiple of 16; 0 without a table
    int interleaved;
    const int* positions;
    const int64_t* slots;
    int num_tokens;
    int n_heads;            // query heads to rotate, 0 without queries
    int n_kv_heads;
    int block_size;
    int num_blocks;
    unsigned int* errors;
};

// Chunks (8 elements, 16 bytes) of item j of a head: whole pairs, so in the
// half layout a chunk and the one rotary_dim / 2 behind it.
struct ItemChunks {
    int a, b;
    bool turn;
};
__device__ __forceinline__ ItemChunks item_chunks(const AppendRopeParams& p, int j) {
    const int half = p.rotary_dim / 16;        // items that are rotated
    if (j < half && !p.interleaved) return {j, j + half, true};
    return {2 * j, 2 * j + 1, j < half};
}

// The cosines and sines of an item's eight pairs.
struct ItemTurn {
    float c[8], s[8];
};
__device__ __forceinline__ void load_turn(const AppendRopeParams& p, int position, int j,
                                          ItemTurn& t) {
    const float* row = p.table + (size_t)position * p.rotary_dim + 8 * j;
    const float* sin_row = row + p.rotary_dim / 2;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<float4*>(t.c + i) = __ldg(reinterpret_cast<const float4*>(row + i));
        *reinterpret_cast<float4*>(t.s + i) = __ldg(reinterpret_cast<const float4*>(sin_row + i));
    }
}

// An item's 16 values in fp32: x[0..7] of chunk a, x[8..15] of chunk b.
template <typename T>
__device__ __forceinline__ void item_values(const uint4& a, const uint4& b, float (&x)[16]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = unpack2<T>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// Pairs (a0, b0) and (a1, b1): one product rounded, the other within the sum, written
// out so that a value does not depend on what the compiler contracts where.
__device__ __forceinline__ void turn_pairs(float& a0, float& b0, float& a1, float& b1, float2 c,
                                           float2 s) {
    const float2 a = make_float2(a0, a1), b = make_float2(b0, b1);
    const float2 x = __ffma2_rn(b, make_float2(-s.x, -s.y), __fmul2_rn(a, c));
    const float2 y = __ffma2_rn(b, c, __fmul2_rn(a, s));
    a0 = x.x;
    a1 = x.y;
    b0 = y.x;
    b1 = y.y;
}

__device__ __forceinline__ void turn_item(float (&x)[16], const ItemTurn& t, int interleaved) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 c = make_float2(t.c[i], t.c[i + 1]), s = make_float2(t.s[i], t.s[i + 1]);
        if (interleaved)
            turn_pairs(x[2 * i], x[2 * i + 1], x[2 * i + 2], x[2 * i + 3], c, s);
        else
            turn_pairs(x[i], x[i + 8], x[i + 1], x[i + 9], c, s);
    }
}

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack_pair<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack_pair<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ void pack_item(const float (&x)[16], uint4& a, uint4& b) {
    a = make_uint4(pack_pair<T>(x[0], x[1]), pack_pair<T>(x[2], x[3]), pack_pair<T>(x[4], x[5]),
                   pack_pair<T>(x[6], x[7]));
    b = make_uint4(pack_pair<T>(x[8], x[9]), pack_pair<T>(x[10], x[11]),
                   pack_pair<T>(x[12], x[13]), pack_pair<T>(x[14], x[15]));
}

// Whether token t is written: its slot in the pool and its position in the
// table (else flagged), both given.
__device__ __forceinline__ bool token_lives(const AppendRopeParams& p, int64_t slot, int position,
                                            bool report) {
    if (slot < 0) return false;
    if (slot >= (int64_t)p.num_blocks * p.block_size) {
        if (report) raise_error(p.errors, PKV_DEVERR_SLOT);
        return false;
    }
    if (p.table && (position < 0 || position >= p.table_rows)) {
        if (report) raise_error(p.errors, PKV_DEVERR_POSITION);
        return false;
    }
    return true;
}

// ------------------------------------------------------------ 16-bit pages
//
// CTA x: a token; its query, key and value heads are kRopeBatch items a thread
// at a time, all loads ahead of the first store (2 / 3 of them: 85 / 80 us
// for 16 prompts of 128-2048 tokens, 32 query and 8 kv heads, 5.9 TB/s; 4 tokens of a
// small model 2.2 us, 250 of 32 heads 4.1).
constexpr int kRopeBatch = 3;

template <int D, typename T>
__global__ void __launch_bounds__(kRopeThreads)
    append_rope_kernel(const __grid_constant__ AppendRopeParams p) {
    constexpr int J = D / 16;                 // items per head
    constexpr int V = D / 8;                  // chunks per head
    const int t = blockIdx.x;
    const int64_t slot = p.slots[t];
    const int position = p.table ? p.positions[t] : 0;
    const int j = threadIdx.x % J;
    const int step = (int)blockDim.x / J;
    const ItemChunks at = item_chunks(p, j);
    const int heads = p.n_heads + 2 * p.n_kv_heads;
    const uint4* q = static_cast<const uint4*>(p.q.p) + (size_t)t * (p.q.stride / 8);
    const uint4* k = static_cast<const uint4*>(p.k.p) + (size_t)t * (p.k.stride / 8);
    const uint4* v = static_cast<const uint4*>(p.v.p) + (size_t)t * (p.v.stride / 8);
    ItemTurn turn;
    bool first = true, live = false;
    for (int h0 = (int)threadIdx.x / J; h0 < heads; h0 += step * kRopeBatch) {
        uint4 a[kRopeBatch], b[kRopeBatch];
#pragma unroll
        for (int i = 0; i < kRopeBatch; ++i) {
            const int h = h0 + i * step;
            if (h >= heads) continue;
            const uint4* row = h < p.n_heads ? q + h * V
                               : h < p.n_heads + p.n_kv_heads
                                   ? k + (h - p.n_heads) * V
                                   : v + (h - p.n_heads - p.n_kv_heads) * V;
            a[i] = __ldcs(row + at.a);
            b[i] = __ldcs(row + at.b);
        }
        if (first) {
            live = token_lives(p, slot, position, threadIdx.x == 0);
            if (live && at.turn) load_turn(p, position, j, turn);
            first = false;
        }
        if (!live) return;
#pragma unroll
        for (int i = 0; i < kRopeBatch; ++i) {
            const int h = h0 + i * step;
            if (h >= heads) continue;
            const int kh = h - p.n_heads;
            const bool value = kh >= p.n_kv_heads;
            if (at.turn && !value) {
                float x[16];
                item_values<T>(a[i], b[i], x);
                turn_item(x, turn, p.interleaved);
                pack_item<T>(x, a[i], b[i]);
            }
            if (kh < 0) {
                uint4* row = static_cast<uint4*>(p.q_out) + (size_t)t * (p.q_out_stride / 8) +
                             h * V;
                row[at.a] = a[i];
                row[at.b] = b[i];
                continue;
            }
            uint4* row = value ? static_cast<uint4*>(p.v_pool) +
                                     ((size_t)slot * p.n_kv_heads + (kh - p.n_kv_heads)) * V
                               : static_cast<uint4*>(p.k_pool) +
                                     ((size_t)slot * p.n_kv_heads + kh) * V;
            row[at.a] = a[i];
            row[at.b] = b[i];
            if (!value && p.k_out) {
                row = static_cast<uint4*>(p.k_out) + (size_t)t * (p.k_out_stride / 8) + kh * V;
                row[at.a] = a[i];
                row[at.b] = b[i];
            }
        }
    }
}

// ------------------------------------------------------------- 8-bit pages
//
// A block's scale covers all its rows of a head, so what is written to a block
// is one unit: a run, tokens that follow one another in the call (but for those left
// out between them, however many) and go to rising rows of one block.  The rows ahead
// of its first one hold tokens and are kept, those behind hold none.  With s(x) the least
// power of two that brings x down to 448 (e4m3's largest), a run sets the scale to s(its
// largest value), or to the old scale if rows are kept and that is larger; kept rows are
// rounded anew where the scale grew.  A power of two costs e4m3 no precision (its numbers
// are spaced relative to their size), and makes the quotients exact and most kept numbers
// survive a new scale unchanged.
//
// CTA x: a window of `window` tokens, whose runs (those that start in it) it takes;
// y: parts of the key and value heads, or of the query heads.  A window is one token,
// or block_size of them: then the rows of its runs are block_size at most but for the
// last run, which goes by itself if it does not fit beside the others.  Runs are found by
// what stands within B tokens of the window; where left-out tokens lie between two of one
// block there, or up to the view's end, the living ones are sought beyond (regather: 250
// tokens padded to 256 4.9 -> 6.0 us, 100 of 256 4.7 -> 5.8, a prompt of 1100 in 2048 11.4
// -> 11.9; 32 query and 8 kv heads of 128).
// A thread holds its items from the one pass over them to the next (the largest
// value, then the codes), while the next part's rows and scales are on their way.
//
// Measured: 8 prompts of 300-2048 tokens, 32 heads of 128, 87-88 us (3.8 TB/s), 16 of 32
// query and 8 kv heads 94 (4.4 TB/s), 4 tokens 3.3 us.  Neither HBM nor the issue slots (62 %
// busy, 300 instructions an item, 20 warps an SM) are full: a step's loads, two barriers
// and codes follow one another.  A warp per run and head, its rows in shared memory and no
// barriers, took 95 us and 6.4 for the 4 tokens; one barrier a step 121; the parts of a
// window side by side in the grid 132; 256 threads 101.

constexpr int kLeastExponent = -117;           // of a scale (a block of zeros)
constexpr int kAppendThreads = 128;
constexpr int kAppendItems = 2;                // items that a thread holds
// CTAs per SM that the registers are shared between (4 / 5 / 6 of them: 16 prompts of 32
// query and 8 kv heads 110 / 98 / 117 us, 8 of 32 heads 99.8 / 98.7 / 118; 6 spill).
constexpr int kAppendCtas = 5;
constexpr int kQ8MaxBlock = 32;                // tokens of a block, and of a window

// Heads that a CTA takes (a power of two): block_size rows of them are kAppendItems a
// thread.
__host__ __device__ constexpr int q8_cta_heads(int D, int block_size) {
    return kAppendThreads * kAppendItems / (block_size * (D / 16));
}

// s(x) of a largest value x >= 0 (finite).
__device__ __forceinline__ float scale_for(float x) {
    const uint32_t bits = __float_as_uint(x);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(e, kLeastExponent);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// 1 / scale where that is exact and a normal number (every scale that an append
// sets), else 0.
__device__ __forceinline__ float exact_inverse(float scale) {
    const uint32_t bits = __float_as_uint(scale), e = bits >> 23;
    return (bits & 0x807fffffu) == 0u && e >= 1 && e <= 253 ? __uint_as_float((254u - e) << 23)
                                                            : 0.f;
}

// Four values to e4m3, to the nearest (ties to even), beyond 448 to 448, NaN to NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    uint32_t w;
    asm("mov.b32 %0, {%1, %2};" : "=r"(w) : "h"(lo), "h"(hi));
    return w;
}

// Two e4m3 to fp32 (exact).
__device__ __forceinline__ float2 unpack_e4m3(uint16_t w) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

struct Q8Row {
    int token;          // of the call
    int run;
    int slot_in_block;
    int position;
};

// Queries of a window of tokens: heads h0 .. h0 + heads - 1.
template <int D, typename T>
__device__ __forceinline__ void append_q8_queries(const AppendRopeParams& p, int w0, int w1, int h0,
                                                  int heads) {
    constexpr int J = D / 16, V = D / 8, kBatch = 4, kStep = kAppendThreads / J;
    const int j = threadIdx.x % J;
    const ItemChunks at = item_chunks(p, j);
    // (token, head) of this thread's next item
    int t = w0 + (int)threadIdx.x / J / heads, h = (int)threadIdx.x / J % heads;
    ItemTurn turn;
    int turn_of = -1;                             // position of `turn`
    while (t < w1) {
        uint4 a[kBatch], b[kBatch];
        int64_t slot[kBatch];
        int position[kBatch], token[kBatch], head[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            token[i] = t;
            head[i] = h0 + h;
            if (t < w1) {
                const uint4* row = static_cast<const uint4*>(p.q.p) +
                                   (size_t)t * (p.q.stride / 8) + head[i] * V;
                a[i] = __ldcs(row + at.a);
                b[i] = __ldcs(row + at.b);
                slot[i] = p.slots[t];
                position[i] = p.table ? p.positions[t] : 0;
            }
            for (h += kStep; h >= heads; h -= heads) ++t;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (token[i] >= w1 || !token_lives(p, slot[i], position[i], false)) continue;
            if (at.turn) {
                if (position[i] != turn_of) {
                    load_turn(p, position[i], j, turn);
                    turn_of = position[i];
                }
                float x[16];
                item_values<T>(a[i], b[i], x);
                turn_item(x, turn, p.interleaved);
                pack_item<T>(x, a[i], b[i]);
            }
            uint4* to = static_cast<uint4*>(p.q_out) + (size_t)token[i] * (p.q_out_stride / 8) +
                        head[i] * V;
            to[at.a] = a[i];
            to[at.b] = b[i];
        }
    }
}

// (out of line: its code would sit in the way of what nearly every block takes)
__device__ __noinline__ float4 divide(float4 x, float by) {
    return make_float4(__fdiv_rn(x.x, by), __fdiv_rn(x.y, by), __fdiv_rn(x.z, by),
                       __fdiv_rn(x.w, by));
}

// The largest finite |x|.
__device__ __forceinline__ float largest(const float (&x)[16]) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i += 2)                                  // (passes NaN over)
        asm("max.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(fabsf(x[i])), "f"(fabsf(x[i + 1])));
    if (top < INFINITY) return top;
    top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fabsf(x[i]) < INFINITY ? fmaxf(top, fabsf(x[i])) : top;
    return top;
}

// The first set bit from `from` on, kAppendThreads if there is none.
__device__ __forceinline__ int next_living(const unsigned* lives, int from) {
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) {
        const int skip = from - 32 * w;
        const unsigned rest = skip >= 32 ? 0u : lives[w] & (0xffffffffu << max(skip, 0));
        if (rest) return 32 * w + __ffs(rest) - 1;
    }
    return kAppendThreads;
}

// Block of token t, -1: left out, or no token.
template <int B>
__device__ __forceinline__ int living_block(const AppendRopeParams& p, long long t) {
    if (t < 0 || t >= p.num_tokens) return -1;
    const int64_t slot = p.slots[t];
    return token_lives(p, slot, p.table ? p.positions[t] : 0, false) ? (int)(slot / B) : -1;
}

// By the whole CTA: whether a token may live (its slot is in the pool) among the
// kLook * kAppendThreads from `at` on, in the direction `way`.
constexpr int kLook = 16;
template <int B>
__device__ __forceinline__ bool group_lives(const AppendRopeParams& p, long long at, int way) {
    const int64_t slots = (int64_t)p.num_blocks * B;
    int64_t slot[kLook];
#pragma unroll
    for (int i = 0; i < kLook; ++i) {
        const long long t = at + way * (i * kAppendThreads + (int)threadIdx.x);
        slot[i] = t >= 0 && t < p.num_tokens ? p.slots[t] : -1;
    }
    bool any = false;
#pragma unroll
    for (int i = 0; i < kLook; ++i) any |= slot[i] >= 0 && slot[i] < slots;
    return __syncthreads_or(any);
}

// The same of all tokens from `at` on.
template <int B>
__device__ __forceinline__ bool rest_lives(const AppendRopeParams& p, long long at, int way) {
    for (; at >= 0 && at < p.num_tokens; at += way * kLook * kAppendThreads)
        if (group_lives<B>(p, at, way)) return true;
    return false;
}

// By the whole CTA: of the tokens that are not left out, tokens[B ..] get the window's
// (their number is returned), tokens[.. B - 1] those ahead of it, the last at B - 1, and
// tokens[B + that number ..] those behind; -1 where there is none.  Ahead and behind they
// are sought, over whatever stands between, until B (B - 1) are found or one of another
// block than the window's first (last): no run goes on beyond.
template <int B>
__device__ __forceinline__ int gather_living(const AppendRopeParams& p, int w0, int w1, int* tokens) {
    __shared__ int s_found;
    __shared__ int s_done;
    const int tid = threadIdx.x, lane = tid & 31;
    const unsigned below = (1u << lane) - 1u;
    if (tid < 3 * B) tokens[tid] = -1;
    const int own = lane < w1 - w0 ? living_block<B>(p, w0 + lane) : -1;   // (32 tokens at most)
    const unsigned living = __ballot_sync(0xffffffffu, own >= 0);
    const int count = __popc(living);
    __syncthreads();
    if (tid < 32 && own >= 0) tokens[B + __popc(living & below)] = w0 + lane;
#pragma unroll 1
    for (int way = -1; way <= 1; way += 2) {
        const int most = way < 0 ? B : B - 1;
        const int edge = __shfl_sync(0xffffffffu, own,
                                     way < 0 ? __ffs(living) - 1 : 31 - __clz(living));
        if (tid == 0) s_found = s_done = 0;
        __syncthreads();
        for (long long at = way < 0 ? w0 - 1LL : w1; at >= 0 && at < p.num_tokens;
             at += way * kLook * kAppendThreads) {
            if (!group_lives<B>(p, at, way)) continue;
            if (tid < 32) {                    // 32 at a time, in order
                int found = s_found;
                bool done = false;
                for (int i = 0; !done && i < kLook * kAppendThreads; i += 32) {
                    const long long t = at + way * (i + lane);
                    const int b = living_block<B>(p, t);
                    const unsigned here = __ballot_sync(0xffffffffu, b >= 0);
                    const int rank = found + __popc(here & below);
                    if (b >= 0 && rank < most)
                        tokens[way < 0 ? B - 1 - rank : B + count + rank] = (int)t;
                    found += __popc(here);
                    done = found >= most || __any_sync(0xffffffffu, b >= 0 && b != edge);
                }
                if (lane == 0) {
                    s_found = found;
                    s_done = done;
                }
            }
            __syncthreads();
            if (s_done) break;
        }
        __syncthreads();
    }
    return count;
}

// By the whole CTA, where tokens around the window are left out: the living tokens of the
// window (their number), gathered with their neighbours where it matters what stands
// between them, that is between two of one block and where nothing in view tells whether
// they stand there.  Thread i looks at token w0 - B + i, at `span` of them; s_blk and s_in
// get what is gathered.  Out of line: batches without padding never come here.
struct Gathered {
    int count;                 // 0: none in the window, -1: nothing is to be gathered
    int token, block, in_block, position;      // this thread's
};
template <int B>
__device__ __noinline__ Gathered regather(const AppendRopeParams& p, int w0, int w1, int span,
                                          int block, int in_block, bool out, int* s_blk, int* s_in) {
    __shared__ unsigned s_lives[kAppendThreads / 32];
    __shared__ int s_tok[3 * B];               // as gather_living lists them
    const int tid = threadIdx.x, t = w0 - B + tid;
    Gathered r = {-1, -1, -1, 0, 0};
    if (out && blockIdx.y == 0 && t >= w0 && t < w1)        // (says what is wrong)
        token_lives(p, p.slots[t], p.table ? p.positions[t] : 0, true);
    const unsigned lives = __ballot_sync(0xffffffffu, block >= 0);
    if ((tid & 31) == 0) s_lives[tid / 32] = lives;
    __syncthreads();
    const int next = next_living(s_lives, tid + 1), first = next_living(s_lives, B);
    if (first >= B + (w1 - w0)) {
        r.count = 0;
        return r;
    }
    bool between = false, behind = false, ahead = false;
    if (block >= 0 && next < kAppendThreads)
        between = next > tid + 1 && s_blk[next] == block;
    else if (block >= 0 && tid >= B && tid + 1 < span && in_block < B - 1) {
        int last = B + (w1 - w0) - 1;          // of the window
        while (!((s_lives[last / 32] >> (last % 32)) & 1u)) --last;
        behind = s_blk[last] == block;
    } else if (out && tid == 0) {
        ahead = s_blk[next] == s_blk[first];
    }
    bool gather = __syncthreads_or(between);
    if (!gather && __syncthreads_or(behind)) gather = rest_lives<B>(p, w0 - B + span, 1);
    if (!gather && __syncthreads_or(ahead)) gather = rest_lives<B>(p, w0 - B - 1LL, -1);
    if (!gather) return r;
    r.count = gather_living<B>(p, w0, w1, s_tok);
    r.token = tid < 3 * B ? s_tok[tid] : -1;
    if (r.token >= 0) {
        const int64_t slot = p.slots[r.token];
        r.position = p.table ? p.positions[r.token] : 0;
        r.block = (int)(slot / B);
        r.in_block = (int)(slot % B);
    }
    if (tid < 3 * B) {
        s_blk[tid] = r.block;
        s_in[tid] = r.in_block;
    }
    __syncthreads();
    return r;
}

template <int D, int B, typename T>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas)
    append_rope_q8_kernel(const __grid_constant__ AppendRopeParams p, int window, int kv_ctas,
                          int cta_parts, int q_heads) {
    constexpr int J = D / 16;
    constexpr int V = D / 8;
    constexpr int HC = q8_cta_heads(D, B);
    constexpr int kPairs = kAppendThreads * kAppendItems / J;   // rows x heads of a CTA
    static_assert(3 * B <= kAppendThreads, "a thread per token around the window");
    __shared__ int s_blk[3 * B];              // block and row of a token's slot, -1: none
    __shared__ int s_in[3 * B];
    __shared__ int s_count[2][kAppendThreads / 32];
    __shared__ Q8Row s_row[2 * kQ8MaxBlock];
    __shared__ int s_first_row[kQ8MaxBlock + 1];  // of a run: its first row in the block
    __shared__ int s_block[kQ8MaxBlock + 1];
    __shared__ int s_last_row;                // of the window's rows: the last run's first
    // of a run and head (in turn): the largest value's bits, then the scale; the old one
    __shared__ uint32_t s_top[2][kPairs];
    __shared__ float s_old[2][kPairs];
    static_assert(kPairs <= kAppendThreads, "a thread per run and head");

    const int tid = threadIdx.x, lane = tid & 31;
    const int j = tid % J;
    const ItemChunks at = item_chunks(p, j);
    const int w0 = blockIdx.x * window, w1 = min(w0 + window, p.num_tokens);
    if ((int)blockIdx.y >= kv_ctas) {
        const int h0 = ((int)blockIdx.y - kv_ctas) * q_heads;
        append_q8_queries<D, T>(p, w0, w1, h0, min(q_heads, p.n_heads - h0));
        return;
    }

    // ---- the tokens around the window: thread i looks at token w0 - B + i
    const int span = min(w1 + B - 1, p.num_tokens) - (w0 - B);
    int t = w0 - B + tid, count = w1 - w0;     // tokens of the window
    bool here = t >= w0 && t < w1;
    int block = -1, in_block = 0, position = 0;
    bool out = false;                          // a token that is left out
    if (tid < span && t >= 0) {
        const int64_t slot = p.slots[t];
        position = p.table ? p.positions[t] : 0;
        out = !token_lives(p, slot, position, false);
        if (!out) {
            block = (int)(slot / B);
            in_block = (int)(slot % B);
        }
    }
    if (tid < 3 * B) {
        s_blk[tid] = block;
        s_in[tid] = in_block;
    }
    if (tid < kPairs) s_top[0][tid] = 0u;
    if (__syncthreads_or(out)) {
        const Gathered g = regather<B>(p, w0, w1, span, block, in_block, out, s_blk, s_in);
        if (g.count == 0) return;
        if (g.count > 0) {
            count = g.count;
            t = g.token;
            here = t >= w0 && t < w1;
            block = g.block;
            in_block = g.in_block;
            position = g.position;
        }
    }
    // distance to the run's first token, -1: in no run
    int back = -1;
    if (block >= 0) {
        // (rising rows of one block: at most B - 1 steps)
        int above = in_block;
        for (back = 0; tid > back && s_blk[tid - back - 1] == block; ++back) {
            const int below = s_in[tid - back - 1];
            if (below >= above) break;
            above = below;
        }
        // a token that follows one of its block but not to a later row ends the run,
        // and what follows it there is in none
        if (tid > back && s_blk[tid - back - 1] == block) {
            back = -1;
            if (here && blockIdx.y == 0) raise_error(p.errors, PKV_DEVERR_SLOT);
        }
    }
    // ---- rows and runs of the window, in order
    const int first = tid - back;                // index of the run's first token
    const bool mine = back >= 0 && first >= B && first < B + count;
    const unsigned rows_here = __ballot_sync(0xffffffffu, mine);
    const unsigned runs_here = __ballot_sync(0xffffffffu, mine && back == 0);
    if (lane == 0) {
        s_count[0][tid / 32] = __popc(rows_here);
        s_count[1][tid / 32] = __popc(runs_here);
    }
    __syncthreads();
    int n_rows = 0, n_runs = 0, row0 = 0, run0 = 0;
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) {
        if (w == tid / 32) {
            row0 = n_rows;
            run0 = n_runs;
        }
        n_rows += s_count[0][w];
        n_runs += s_count[1][w];
    }
    if (mine) {
        const unsigned upto = 0xffffffffu >> (31 - lane);      // lanes 0 .. lane
        const int r = row0 + __popc(rows_here & upto) - 1, run = run0 + __popc(runs_here & upto) - 1;
        s_row[r] = {t, run, in_block, position};
        if (back == 0) {
            s_first_row[run] = in_block;
            s_block[run] = block;
            if (run == n_runs - 1) s_last_row = r;
        }
    }
    __syncthreads();
    if (n_rows == 0) return;

    // ---- parts of HC heads, each in one batch, or two with the last run by itself
    const int n_slots = 2 * p.n_kv_heads;                    // head slots: keys, then values
    const bool split = n_rows > B;
    const int batches = split ? 2 : 1;
    const int n_parts = min(cta_parts, (n_slots + HC - 1) / HC - (int)blockIdx.y * cta_parts);
    const int n_steps = n_parts * batches;
    // item n of this thread: row r0 + n * kRowStep of the batch, head h of the part
    constexpr int kRowStep = kAppendThreads / (J * HC);
    static_assert(kRowStep >= 1 && kRowStep * kAppendItems == B, "items");
    const int h = tid / J % HC, r0 = tid / (J * HC);
    struct Step {
        int hs0;                    // first head slot
        int row_lo, row_hi, run_lo, run_hi;
    };
    auto step_at = [&](int i) -> Step {
        const int batch = i % batches;
        Step s;
        s.hs0 = ((int)blockIdx.y * cta_parts + i / batches) * HC;
        s.row_lo = batch ? s_last_row : 0;
        s.row_hi = split && !batch ? s_last_row : n_rows;
        s.run_lo = batch ? n_runs - 1 : 0;
        s.run_hi = split && !batch ? n_runs - 1 : n_runs;
        return s;
    };
    uint4 a[kAppendItems], b[kAppendItems];
    float old = 0.f;                // thread e: old scale of run e / HC, head e % HC
    auto fetch = [&](const Step& s) {
        const int hs = s.hs0 + h;
        const bool key = hs < p.n_kv_heads;
        const uint4* const from = static_cast<const uint4*>(key ? p.k.p : p.v.p) +
                                  (key ? hs : hs - p.n_kv_heads) * V;
        const size_t stride = (size_t)(key ? p.k.stride : p.v.stride) / 8;
#pragma unroll
        for (int n = 0; n < kAppendItems; ++n) {
            const int r = s.row_lo + r0 + n * kRowStep;
            if (hs >= n_slots || r >= s.row_hi) continue;
            const uint4* row = from + s_row[r].token * stride;
            a[n] = __ldcs(row + at.a);
            b[n] = __ldcs(row + at.b);
        }
        const int run = s.run_lo + tid / HC, es = s.hs0 + tid % HC;
        old = 0.f;
        if (run < s.run_hi && es < n_slots && s_first_row[run] > 0)
            old = (es < p.n_kv_heads ? p.k_scale + es : p.v_scale + (es - p.n_kv_heads))
                [(size_t)s_block[run] * p.n_kv_heads];
    };
    Step now = step_at(0);
    fetch(now);
    for (int i = 0; i < n_steps; ++i) {
        uint32_t* const top = s_top[i & 1];
        const int hs = now.hs0 + h;
        const bool key = hs < p.n_kv_heads, real = hs < n_slots;
        const int kvh = key ? hs : hs - p.n_kv_heads;
        // ---- values, rotated, and the largest of every run and head
        float x[kAppendItems][16], most[kAppendItems] = {};
        unsigned lives = 0u;                  // items that are written
#pragma unroll
        for (int n = 0; n < kAppendItems; ++n) {
            const int r = now.row_lo + r0 + n * kRowStep;
            if (!real || r >= now.row_hi) continue;
            lives |= 1u << n;
            item_values<T>(a[n], b[n], x[n]);
            if (key && at.turn) {
                ItemTurn turn;
                load_turn(p, s_row[r].position, j, turn);
                turn_item(x[n], turn, p.interleaved);
            }
            if (key && p.k_out) {
                if (at.turn) pack_item<T>(x[n], a[n], b[n]);
                uint4* to = static_cast<uint4*>(p.k_out) +
                            (size_t)s_row[r].token * (p.k_out_stride / 8) + kvh * V;
                to[at.a] = a[n];
                to[at.b] = b[n];
            }
            most[n] = largest(x[n]);
        }
        // (a head's items are on J neighbouring lanes)
#pragma unroll
        for (int n = 0; n < kAppendItems; ++n) {
#pragma unroll
            for (int off = 1; off < J; off <<= 1)
                most[n] = fmaxf(most[n], __shfl_xor_sync(0xffffffffu, most[n], off));
            if (j == 0 && ((lives >> n) & 1u))
                atomicMax(&top[(s_row[now.row_lo + r0 + n * kRowStep].run - now.run_lo) * HC + h],
                          __float_as_uint(most[n]));
        }
        const float was = old;
        const Step next = step_at(min(i + 1, n_steps - 1));
        if (i + 1 < n_steps) fetch(next);
        __syncthreads();
        // ---- scales
        const int pairs = (now.run_hi - now.run_lo) * HC;
        if (tid < pairs && now.hs0 + tid % HC < n_slots) {
            const int run = now.run_lo + tid / HC, es = now.hs0 + tid % HC;
            const float scale = fmaxf(scale_for(__uint_as_float(top[tid])), was);
            float* to = es < p.n_kv_heads ? p.k_scale + es : p.v_scale + (es - p.n_kv_heads);
            if (s_first_row[run] == 0 || scale != was)
                to[(size_t)s_block[run] * p.n_kv_heads] = scale;
            top[tid] = __float_as_uint(scale);
            s_old[i & 1][tid] = was;
        }
        if (tid < kPairs) s_top[(i + 1) & 1][tid] = 0u;
        __syncthreads();
        // ---- new rows
        unsigned char* const page0 = static_cast<unsigned char*>(key ? p.k_pool : p.v_pool) +
                                     (size_t)kvh * D;
#pragma unroll
        for (int n = 0; n < kAppendItems; ++n) {
            if (!((lives >> n) & 1u)) continue;
            const Q8Row r = s_row[now.row_lo + r0 + n * kRowStep];
            const float scale = __uint_as_float(top[(r.run - now.run_lo) * HC + h]);
            const float inv = exact_inverse(scale);
            if (inv > 0.f) {
#pragma unroll
                for (int c = 0; c < 16; c += 2) {
                    const float2 y = __fmul2_rn(make_float2(x[n][c], x[n][c + 1]),
                                                make_float2(inv, inv));
                    x[n][c] = y.x;
                    x[n][c + 1] = y.y;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                    const float4 y = divide(
                        make_float4(x[n][c], x[n][c + 1], x[n][c + 2], x[n][c + 3]), scale);
                    x[n][c] = y.x;
                    x[n][c + 1] = y.y;
                    x[n][c + 2] = y.z;
                    x[n][c + 3] = y.w;
                }
            }
            unsigned char* row = page0 + ((size_t)s_block[r.run] * B + r.slot_in_block) *
                                             p.n_kv_heads * D;
            *reinterpret_cast<uint2*>(row + at.a * 8) =
                make_uint2(pack_e4m3(x[n][0], x[n][1], x[n][2], x[n][3]),
                           pack_e4m3(x[n][4], x[n][5], x[n][6], x[n][7]));
            *reinterpret_cast<uint2*>(row + at.b * 8) =
                make_uint2(pack_e4m3(x[n][8], x[n][9], x[n][10], x[n][11]),
                           pack_e4m3(x[n][12], x[n][13], x[n][14], x[n][15]));
        }
        // ---- kept rows of a scale that grew, a warp per run and head
        for (int e = tid / 32; e < pairs; e += kAppendThreads / 32) {
            const int run = now.run_lo + e / HC, es = now.hs0 + e % HC;
            const int kept = s_first_row[run];
            if (es >= n_slots || kept == 0) continue;
            const float scale = __uint_as_float(top[e]), from = s_old[i & 1][e];
            if (scale == from) continue;
            const float ratio = __fdiv_rn(from, scale);
            const bool of_keys = es < p.n_kv_heads;
            unsigned char* page = static_cast<unsigned char*>(of_keys ? p.k_pool : p.v_pool) +
                                  ((size_t)s_block[run] * B * p.n_kv_heads +
                                   (of_keys ? es : es - p.n_kv_heads)) * D;
            for (int c = lane; c < kept * (D / 16); c += 32) {
                uint4* at16 = reinterpret_cast<uint4*>(page + (size_t)(c / (D / 16)) *
                                                                  p.n_kv_heads * D) +
                              c % (D / 16);
                const uint4 codes = *at16;
                const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
                uint32_t anew[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 lo = unpack_e4m3((uint16_t)w[k]);
                    const float2 hi = unpack_e4m3((uint16_t)(w[k] >> 16));
                    anew[k] = pack_e4m3(lo.x * ratio, lo.y * ratio, hi.x * ratio, hi.y * ratio);
                }
                *at16 = make_uint4(anew[0], anew[1], anew[2], anew[3]);
            }
        }
        now = next;
    }
}

// ------------------------------------------------------------------- table

struct RopeTableParams {
    float* table;           // [positions, 2 pairs]
    int positions;
    int pairs;
    float factor;
    double freq[64];        // angle of pair i at position t: t * freq[i]
};

// Angles and their functions in 64 bits: at position 131072 an fp32 angle is
// off by up to 2^-8, more than bf16's half step of a cosine.
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ RopeTableParams p) {
    const long long total = (long long)p.positions * p.pairs;
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
         i += (long long)gridDim.x * blockDim.x) {
        const int t = (int)(i / p.pairs), k = (int)(i % p.pairs);
        double s, c;
        sincos(t * p.freq[k], &s, &c);
        float* row = p.table + (size_t)t * 2 * p.pairs;
        row[k] = (float)(c * p.factor);
        row[p.pairs + k] = (float)(s * p.factor);
    }
}

}  // namespace pkv
