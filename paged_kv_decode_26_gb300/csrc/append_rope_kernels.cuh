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

// (one product rounded, the other within the sum, written out so that a value
// does not depend on what the compiler contracts where)
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
    const float x = __fmaf_rn(a, c, -__fmul_rn(b, s)), y = __fmaf_rn(a, s, __fmul_rn(b, c));
    a = x;
    b = y;
}

__device__ __forceinline__ void turn_item(float (&x)[16], const ItemTurn& t, int interleaved) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(x[2 * i], x[2 * i + 1], t.c[i], t.s[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(x[i], x[i + 8], t.c[i], t.s[i]);
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
// at a time, all loads ahead of the first store.
constexpr int kRopeBatch = 2;

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
// is one unit: a run, tokens that follow one another in the call and go to
// rising rows of one block.  The rows ahead of its first one hold tokens and are
// kept, those behind hold none.  With s(x) the least power of two that brings x
// down to 448 (e4m3's largest), a run sets the scale to s(its largest value), or
// to the old scale if rows are kept and that is larger; kept rows are rounded
// anew where the scale grew.  A power of two costs e4m3 no precision (its
// numbers are spaced relative to their size), and makes the quotients exact and
// most kept numbers survive a new scale unchanged.
//
// CTA x: a window of `window` tokens, whose runs (those that start in it) it
// takes in turn, as many at a time as fit block_size rows; y: a part of the key
// and value heads, then parts of the query heads.

constexpr float kE4m3Max = 448.f;
constexpr int kLeastExponent = -117;           // of a scale (a block of zeros)
constexpr int kQ8Items = 4;                    // items that a thread holds
constexpr int kQ8Window = 32;                  // most tokens of a window
constexpr int kQ8MaxBlock = 32;

// Heads that a CTA takes: block_size rows of them are kQ8Items a thread.
__host__ __device__ constexpr int q8_cta_heads(int D, int block_size) {
    return kRopeThreads * kQ8Items / (block_size * (D / 16));
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
    return (uint32_t)lo | (uint32_t)hi << 16;
}

// Two e4m3 to fp32 (exact).
__device__ __forceinline__ float2 unpack_e4m3(uint16_t w) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

struct Q8Row {
    int token;          // of the call
    int run;            // index of the row's run in the batch
    int64_t slot;
    int position;
};

template <int D, typename T>
__global__ void __launch_bounds__(kRopeThreads)
    append_rope_q8_kernel(const __grid_constant__ AppendRopeParams p, int window, int kv_parts,
                          int cta_heads, int q_heads) {
    constexpr int J = D / 16;
    constexpr int V = D / 8;
    constexpr int kSpan = kQ8MaxBlock + kQ8Window + kQ8MaxBlock;
    __shared__ int s_blk[kSpan];              // block and row of a token's slot, -1: none
    __shared__ int s_in[kSpan];
    __shared__ int s_pos[kSpan];
    __shared__ int s_head[kSpan];             // distance to the run's first token, -1: in none
    __shared__ Q8Row s_row[kQ8MaxBlock];
    __shared__ int s_first_row[kQ8MaxBlock];  // of a run: its first row in the block
    __shared__ int s_block[kQ8MaxBlock];
    // of a run and head: the largest value's bits, then the scale
    __shared__ uint32_t s_top[kRopeThreads * kQ8Items / 4];
    __shared__ float s_old[kRopeThreads * kQ8Items / 4];
    __shared__ int s_rows, s_runs, s_next;

    const int tid = threadIdx.x, B = p.block_size;
    const int j = tid % J;
    const ItemChunks at = item_chunks(p, j);
    const int w0 = blockIdx.x * window, w1 = min(w0 + window, p.num_tokens);

    if ((int)blockIdx.y >= kv_parts) {
        // ---- queries
        const int h0 = ((int)blockIdx.y - kv_parts) * q_heads;
        const int heads = min(q_heads, p.n_heads - h0);
        const int items = (w1 - w0) * heads * J;
        for (int e = tid; e < items; e += kRopeThreads) {
            const int h = h0 + e / J % heads, t = w0 + e / J / heads;
            const uint4* row = static_cast<const uint4*>(p.q.p) + (size_t)t * (p.q.stride / 8) +
                               h * V;
            uint4 a = __ldcs(row + at.a), b = __ldcs(row + at.b);
            const int64_t slot = p.slots[t];
            const int position = p.table ? p.positions[t] : 0;
            if (!token_lives(p, slot, position, false)) continue;
            if (at.turn) {
                float x[16];
                item_values<T>(a, b, x);
                ItemTurn turn;
                load_turn(p, position, j, turn);
                turn_item(x, turn, p.interleaved);
                pack_item<T>(x, a, b);
            }
            uint4* to = static_cast<uint4*>(p.q_out) + (size_t)t * (p.q_out_stride / 8) + h * V;
            to[at.a] = a;
            to[at.b] = b;
        }
        return;
    }

    // ---- the tokens around the window: index i is token w0 - B + i
    const int span = min(w1 + B - 1, p.num_tokens) - (w0 - B), shift = B == 16 ? 4 : 5;
    for (int i = tid; i < span; i += kRopeThreads) {
        const int t = w0 - B + i;
        const int64_t slot = t >= 0 ? p.slots[t] : -1;
        const int position = t >= 0 && p.table ? p.positions[t] : 0;
        const bool here = blockIdx.y == 0 && t >= w0 && t < w1;
        if (here) token_lives(p, slot, position, true);      // (says what is wrong)
        const bool in_pool = slot >= 0 && slot < (int64_t)p.num_blocks * B;
        s_blk[i] = in_pool ? (int)(slot >> shift) : -1;
        s_in[i] = (int)(slot & (B - 1));
        s_pos[i] = position;
    }
    __syncthreads();
    for (int i = tid; i < span; i += kRopeThreads) {
        const int block = s_blk[i];
        int back = block < 0 ? -1 : 0;
        if (block >= 0) {
            // (rising rows of one block: at most B - 1 steps)
            while (i > back && s_blk[i - back - 1] == block && s_in[i - back] > s_in[i - back - 1])
                ++back;
            // a token that follows one of its block but not to a later row ends
            // the run, and what follows it there is in none
            if (i > back && s_blk[i - back - 1] == block) {
                back = -1;
                const int t = w0 - B + i;
                if (blockIdx.y == 0 && t >= w0 && t < w1) raise_error(p.errors, PKV_DEVERR_SLOT);
            }
        }
        s_head[i] = back;
    }
    __syncthreads();

    const int hs0 = (int)blockIdx.y * cta_heads;             // head slots: keys, then values
    const int heads = min(cta_heads, 2 * p.n_kv_heads - hs0);
    int next = B;                                            // token index to go on at
    while (next < B + (w1 - w0)) {
        // ---- whole runs, up to B rows
        if (tid == 0) {
            int rows = 0, runs = 0, i = next;
            for (; i < span; ++i) {
                const int back = s_head[i];
                if (back < 0) {
                    if (i >= B + (w1 - w0)) break;
                    continue;
                }
                if (back == 0) {
                    if (i >= B + (w1 - w0)) break;           // another window's
                    int n = 1;
                    while (i + n < span && s_head[i + n] == n) ++n;
                    if (rows + n > B) break;
                    s_first_row[runs] = s_in[i];
                    s_block[runs] = s_blk[i];
                    ++runs;
                } else if (i - back < next) {
                    continue;                                // an earlier window's run
                }
                s_row[rows].token = w0 - B + i;
                s_row[rows].run = runs - 1;
                s_row[rows].slot = ((int64_t)s_blk[i] << shift) + s_in[i];
                s_row[rows].position = s_pos[i];
                ++rows;
            }
            s_rows = rows;
            s_runs = runs;
            s_next = i;
        }
        __syncthreads();
        const int rows = s_rows, runs = s_runs;
        next = s_next;
        const int pairs = runs * heads;
        for (int e = tid; e < pairs; e += kRopeThreads) {
            const int hs = hs0 + e % heads;
            const float* scale = hs < p.n_kv_heads ? p.k_scale + hs : p.v_scale + (hs - p.n_kv_heads);
            s_top[e] = 0u;
            s_old[e] = s_first_row[e / heads] > 0
                           ? scale[(size_t)s_block[e / heads] * p.n_kv_heads]
                           : 0.f;
        }
        __syncthreads();
        // ---- values, rotated, and the largest of every run and head
        float x[kQ8Items][16];
        const int items = rows * heads * J;
#pragma unroll
        for (int n = 0; n < kQ8Items; ++n) {
            const int e = tid + n * kRopeThreads;
            if (e >= items) continue;
            const int h = e / J % heads, hs = hs0 + h;
            const Q8Row& r = s_row[e / J / heads];
            const bool key = hs < p.n_kv_heads;
            const RopeSource& src = key ? p.k : p.v;
            const uint4* row = static_cast<const uint4*>(src.p) +
                               (size_t)r.token * (src.stride / 8) +
                               (key ? hs : hs - p.n_kv_heads) * V;
            uint4 a = __ldcs(row + at.a), b = __ldcs(row + at.b);
            item_values<T>(a, b, x[n]);
            const bool lives = !p.table || (r.position >= 0 && r.position < p.table_rows);
            float top = 0.f;
            if (lives) {
                if (key && at.turn) {
                    ItemTurn turn;
                    load_turn(p, r.position, j, turn);
                    turn_item(x[n], turn, p.interleaved);
                }
                if (key && p.k_out) {
                    if (at.turn) pack_item<T>(x[n], a, b);
                    uint4* to = static_cast<uint4*>(p.k_out) +
                                (size_t)r.token * (p.k_out_stride / 8) + hs * V;
                    to[at.a] = a;
                    to[at.b] = b;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float y = fabsf(x[n][i]);
                    top = fmaxf(top, y <= 3.4028234e38f ? y : 0.f);   // (of finite ones)
                }
            }
            // (a head's items are on J neighbouring lanes)
            const unsigned group = (unsigned)((1u << J) - 1u) << (tid % 32 / J * J);
            const uint32_t bits = __reduce_max_sync(group, __float_as_uint(top));
            if (j == 0) atomicMax(&s_top[r.run * heads + h], bits);
        }
        __syncthreads();
        // ---- scales
        for (int e = tid; e < pairs; e += kRopeThreads) {
            const int run = e / heads, hs = hs0 + e % heads;
            const float old = s_old[e];
            const float scale = fmaxf(scale_for(__uint_as_float(s_top[e])), old);
            float* to = hs < p.n_kv_heads ? p.k_scale + hs : p.v_scale + (hs - p.n_kv_heads);
            if (s_first_row[run] == 0 || scale != old)
                to[(size_t)s_block[run] * p.n_kv_heads] = scale;
            s_top[e] = __float_as_uint(scale);
        }
        __syncthreads();
        // ---- new rows
#pragma unroll
        for (int n = 0; n < kQ8Items; ++n) {
            const int e = tid + n * kRopeThreads;
            if (e >= items) continue;
            const int h = e / J % heads, hs = hs0 + h;
            const Q8Row& r = s_row[e / J / heads];
            if (p.table && (r.position < 0 || r.position >= p.table_rows)) continue;
            const float scale = __uint_as_float(s_top[r.run * heads + h]);
            const float inv = exact_inverse(scale);
            if (inv > 0.f) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[n][i] *= inv;
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[n][i] = __fdiv_rn(x[n][i], scale);
            }
            const bool key = hs < p.n_kv_heads;
            unsigned char* row = static_cast<unsigned char*>(key ? p.k_pool : p.v_pool) +
                                 ((size_t)r.slot * p.n_kv_heads +
                                  (key ? hs : hs - p.n_kv_heads)) * D;
            *reinterpret_cast<uint2*>(row + at.a * 8) =
                make_uint2(pack_e4m3(x[n][0], x[n][1], x[n][2], x[n][3]),
                           pack_e4m3(x[n][4], x[n][5], x[n][6], x[n][7]));
            *reinterpret_cast<uint2*>(row + at.b * 8) =
                make_uint2(pack_e4m3(x[n][8], x[n][9], x[n][10], x[n][11]),
                           pack_e4m3(x[n][12], x[n][13], x[n][14], x[n][15]));
        }
        // ---- kept rows of a scale that grew, a warp per run and head
        for (int e = tid / 32; e < pairs; e += kRopeThreads / 32) {
            const int run = e / heads, hs = hs0 + e % heads;
            const float scale = __uint_as_float(s_top[e]), old = s_old[e];
            const int kept = s_first_row[run];
            if (kept == 0 || scale == old) continue;
            const float ratio = __fdiv_rn(old, scale);
            const bool key = hs < p.n_kv_heads;
            unsigned char* page = static_cast<unsigned char*>(key ? p.k_pool : p.v_pool) +
                                  ((size_t)s_block[run] * B * p.n_kv_heads +
                                   (key ? hs : hs - p.n_kv_heads)) * D;
            for (int c = tid % 32; c < kept * (D / 16); c += 32) {
                uint4* at16 = reinterpret_cast<uint4*>(page + (size_t)(c / (D / 16)) *
                                                                  p.n_kv_heads * D) +
                              c % (D / 16);
                const uint4 was = *at16;
                const uint32_t w[4] = {was.x, was.y, was.z, was.w};
                uint32_t now[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 lo = unpack_e4m3((uint16_t)w[i]);
                    const float2 hi = unpack_e4m3((uint16_t)(w[i] >> 16));
                    now[i] = pack_e4m3(lo.x * ratio, lo.y * ratio, hi.x * ratio, hi.y * ratio);
                }
                *at16 = make_uint4(now[0], now[1], now[2], now[3]);
            }
        }
        __syncthreads();
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
