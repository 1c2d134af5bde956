// append_rope_capi.cu -- the C ABI's appends that rotate on the way
// (kv_append_rope, kv_append_rope_q8) and their table (pkv_rope_table):
// validation and launches.  Declarations and contracts: pagedkv.h.
#include <cudaTypedefs.h>

#include <cmath>
#include <cstring>

#include "append_rope_kernels.cuh"
#include "capi_host.h"
#include "pieces_host.h"

using namespace pkv::host;

namespace {

struct Span {
    uintptr_t from, to;
    bool meets(const Span& o) const { return from < o.to && o.from < to; }
};

// Bytes between the first and the last element of `tokens` rows.
Span rows_span(const void* p, int64_t stride, int tokens, int heads, int head_dim) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint64_t row = (uint64_t)heads * head_dim;
    return {a, a + 2 * ((uint64_t)(tokens - 1) * (uint64_t)stride + row)};
}

// Rows of one tensor side by side: a's `an` elements a token, then b's, or the other way.
bool side_by_side(const void* a, int64_t a_stride, int64_t an, const void* b, int64_t b_stride,
                  int64_t bn) {
    if (a_stride != b_stride) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    const uint64_t xn = 2 * (uint64_t)an, yn = 2 * (uint64_t)bn, row = 2 * (uint64_t)a_stride;
    return x < y ? y - x >= xn && y - x + yn <= row : x - y >= yn && x - y + xn <= row;
}

Span pool_span(const void* p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + bytes};
}

pkv_status check_rows(const void* p, int64_t stride, int heads, int head_dim, const char* what) {
    if (!p) return invalid(what);
    if (!aligned16(p)) return invalid("q, k, v and their outputs must be 16-byte aligned");
    if (stride < (int64_t)heads * head_dim || stride % 8)
        return invalid("token strides: multiples of 8 elements, no less than a token's heads");
    if (stride > (int64_t)1 << 40) return unsupported("token stride");
    return PKV_OK;
}

// What both appends check; fills p.
pkv_status fill_append(pkv::AppendRopeParams* pp, int es, void* k_pool, void* v_pool, const void* k,
                       int64_t k_stride, const void* v, int64_t v_stride, pkv_dtype dtype,
                       const int64_t* slot_mapping, const int32_t* positions,
                       const float* rope_table, int table_positions, int rotary_dim,
                       int interleaved, const void* q, int64_t q_stride, void* q_out,
                       int64_t q_out_stride, void* k_out, int64_t k_out_stride, int num_tokens,
                       int n_heads, int n_kv_heads, int head_dim, int block_size, int num_blocks) {
    if (num_tokens < 0 || n_kv_heads <= 0 || block_size <= 0 || num_blocks < 0 || n_heads < 0)
        return invalid("sizes");
    if (dtype != PKV_F16 && dtype != PKV_BF16) return unsupported("dtype must be F16 or BF16");
    if (head_dim != 64 && head_dim != 128) return unsupported("head_dim 64 or 128");
    if (n_kv_heads > 4096 || n_heads > 4096) return unsupported("more than 4096 heads");
    if (rope_table) {
        if (rotary_dim <= 0 || rotary_dim > head_dim || rotary_dim % 16)
            return invalid("rotary_dim must be a multiple of 16, at most head_dim");
        if (table_positions < 0) return invalid("table_positions");
        if (!aligned16(rope_table)) return invalid("rope_table must be 16-byte aligned");
    } else if (q || q_out || k_out) {
        return invalid("q, q_out and k_out without a rope_table");
    }
    if ((q == nullptr) != (q_out == nullptr)) return invalid("q and q_out: both or neither");
    if (q && n_heads <= 0) return invalid("n_heads");
    if (num_tokens == 0) return PKV_OK;
    if (!slot_mapping || (num_blocks > 0 && (!k_pool || !v_pool))) return invalid("NULL pointer");
    if (rope_table && !positions) return invalid("positions is NULL");
    if (!aligned16(k_pool) || !aligned16(v_pool))
        return invalid("k_pool and v_pool must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(slot_mapping) & 7u) != 0)
        return invalid("slot_mapping must be 8-byte aligned");
    if (!aligned4(positions)) return invalid("positions must be 4-byte aligned");
    pkv_status st;
    if ((st = check_rows(k, k_stride, n_kv_heads, head_dim, "k is NULL")) != PKV_OK) return st;
    if ((st = check_rows(v, v_stride, n_kv_heads, head_dim, "v is NULL")) != PKV_OK) return st;
    const size_t pool = (size_t)num_blocks * block_size * n_kv_heads * head_dim * es;
    const Span pools[2] = {pool_span(k_pool, pool), pool_span(v_pool, pool)};
    Span in[3] = {rows_span(k, k_stride, num_tokens, n_kv_heads, head_dim),
                  rows_span(v, v_stride, num_tokens, n_kv_heads, head_dim), {0, 0}};
    if (q) {
        if ((st = check_rows(q, q_stride, n_heads, head_dim, "q is NULL")) != PKV_OK) return st;
        in[2] = rows_span(q, q_stride, num_tokens, n_heads, head_dim);
    }
    if (pool > 0 && pools[0].meets(pools[1])) return invalid("k_pool and v_pool overlap");
    // an output is its own input in place, or apart from all that is read
    Span out[2] = {{0, 0}, {0, 0}};
    for (int i = 0; i < 2; ++i) {
        void* o = i ? k_out : q_out;
        if (!o) continue;
        const int64_t stride = i ? k_out_stride : q_out_stride;
        const int heads = i ? n_kv_heads : n_heads;
        if ((st = check_rows(o, stride, heads, head_dim, "")) != PKV_OK) return st;
        out[i] = rows_span(o, stride, num_tokens, heads, head_dim);
        const bool in_place = o == (i ? k : q) && stride == (i ? k_stride : q_stride);
        const void* const from[3] = {k, v, q};
        const int64_t strides[3] = {k_stride, v_stride, q_stride};
        for (int n = 0; n < 3; ++n) {
            if (!out[i].meets(in[n]) || (in_place && n == (i ? 0 : 2))) continue;
            // (in place, beside the others in one tensor)
            if (!in_place || !side_by_side(o, stride, (int64_t)heads * head_dim, from[n], strides[n],
                                           (int64_t)(n == 2 ? n_heads : n_kv_heads) * head_dim))
                return invalid("q_out and k_out: in place, or apart from q, k and v");
        }
        for (const Span& s : pools)
            if (pool > 0 && out[i].meets(s)) return invalid("q_out and k_out overlap a pool");
    }
    if (q_out && k_out && out[0].meets(out[1]) &&
        !side_by_side(q_out, q_out_stride, (int64_t)n_heads * head_dim, k_out, k_out_stride,
                      (int64_t)n_kv_heads * head_dim))
        return invalid("q_out and k_out overlap");
    for (const Span& s : in)
        for (const Span& w : pools)
            if (pool > 0 && s.from != s.to && s.meets(w)) return invalid("q, k or v overlaps a pool");
    pkv::AppendRopeParams& p = *pp;
    p.q = {q, q_stride};
    p.k = {k, k_stride};
    p.v = {v, v_stride};
    p.q_out = q_out;
    p.q_out_stride = q_out_stride;
    p.k_out = k_out;
    p.k_out_stride = k_out_stride;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.table = rope_table;
    p.table_rows = table_positions;
    p.rotary_dim = rope_table ? rotary_dim : 0;
    p.interleaved = interleaved != 0;
    p.positions = positions;
    p.slots = slot_mapping;
    p.num_tokens = num_tokens;
    p.n_heads = q ? n_heads : 0;
    p.n_kv_heads = n_kv_heads;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    return PKV_OK;
}

int round_up(int x, int m) { return (x + m - 1) / m * m; }

template <int D, typename T>
void launch_append(const pkv::AppendRopeParams& p, cudaStream_t stream) {
    // kRopeBatch items a thread in one go, up to kRopeThreads threads
    const int items = (p.n_heads + 2 * p.n_kv_heads) * (D / 16);
    const int threads = round_up((items + pkv::kRopeBatch - 1) / pkv::kRopeBatch, 32);
    pkv::append_rope_kernel<D, T>
        <<<(unsigned)p.num_tokens, threads < pkv::kRopeThreads ? threads : pkv::kRopeThreads, 0,
           stream>>>(p);
}

// CTAs per SM up to which a CTA takes one token, and from which windows of block_size
// tokens, where one takes several parts of the heads.
// Windows, one token a CTA / windows, us: decode tokens of 32 query and 8 kv heads of 128,
// pages of 16 (9 CTAs a token), 64 3.7 / 4.5, 96 5.4 / 4.6, 512 14 / 5.5; 32 of 32 heads,
// pages of 32 (65 a token), 8 3.4 / 3.3, 16 5.3 / 3.5, 160 26 / 5.3; 8 of 1 head of 64
// (2 a token), 448 3.8 / 5.4, 1024 7.0 / 5.5.  Of 540 sizes the rule takes 0.5 % longer in
// sum than the better of both each (at 5 a SM 1.5 %, at 7 and 8 0.4 and 0.5 %).
// Several parts (4 / 6 / 9 / 14): 8 MHA prompts 97 / 85 / 87 / 91 us, 16 GQA prompts 94 /
// 94 / 98 / 98.
constexpr int kQ8CtasPerSm = 6;

template <int D, int B, typename T>
void launch_append_q8_of(const pkv::AppendRopeParams& p, int sm_count, cudaStream_t stream) {
    constexpr int J = D / 16, heads = pkv::q8_cta_heads(D, B);
    const int parts = (2 * p.n_kv_heads + heads - 1) / heads;
    // query heads and parts of them, at `tokens` a CTA
    auto heads_of = [&](int tokens) {
        const int most = pkv::kAppendThreads * pkv::kAppendItems / (tokens * J);
        return most < 1 ? 1 : (most > p.n_heads ? p.n_heads : most);
    };
    auto parts_of = [&](int tokens) {
        const int n = heads_of(tokens);
        return n > 0 ? (p.n_heads + n - 1) / n : 0;
    };
    const long long enough = (long long)kQ8CtasPerSm * sm_count;
    const int window = (long long)p.num_tokens * (parts + parts_of(1)) > enough ? B : 1;
    const int windows = (p.num_tokens + window - 1) / window;
    // parts one after the other in a CTA, as long as there are enough CTAs
    int cta_parts = (int)((long long)windows * parts / enough);
    cta_parts = cta_parts < 1 ? 1 : (cta_parts > parts ? parts : cta_parts);
    const int kv_ctas = (parts + cta_parts - 1) / cta_parts;
    const int q_heads = heads_of(window);
    const dim3 grid((unsigned)windows, (unsigned)(kv_ctas + parts_of(window)));
    pkv::append_rope_q8_kernel<D, B, T>
        <<<grid, pkv::kAppendThreads, 0, stream>>>(p, window, kv_ctas, cta_parts, q_heads);
}

template <int D, typename T>
void launch_append_q8(const pkv::AppendRopeParams& p, int sm_count, cudaStream_t stream) {
    p.block_size == 16 ? launch_append_q8_of<D, 16, T>(p, sm_count, stream)
                       : launch_append_q8_of<D, 32, T>(p, sm_count, stream);
}

}  // namespace

extern "C" {

PKV_API pkv_status pkv_rope_table(float* table, int num_positions, int rotary_dim,
                                  const double* inv_freq, float factor, void* stream) {
    if (num_positions < 0) return invalid("sizes");
    if (rotary_dim <= 0 || rotary_dim > 128 || rotary_dim % 16)
        return invalid("rotary_dim must be a multiple of 16, at most 128");
    if (!std::isfinite(factor)) return invalid("factor is not finite");
    if (!inv_freq) return invalid("inv_freq is NULL");
    pkv::RopeTableParams p;
    std::memset(&p, 0, sizeof(p));
    for (int i = 0; i < rotary_dim / 2; ++i) {
        if (!std::isfinite(inv_freq[i])) return invalid("inv_freq is not finite");
        p.freq[i] = inv_freq[i];
    }
    if (num_positions == 0) return PKV_OK;
    if (!table) return invalid("table is NULL");
    if (!aligned16(table)) return invalid("table must be 16-byte aligned");
    DeviceInfo* dev = nullptr;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    p.table = table;
    p.positions = num_positions;
    p.pairs = rotary_dim / 2;
    p.factor = factor;
    const long long ctas = ((long long)num_positions * p.pairs + 255) / 256;
    const long long most = 8LL * dev->sm_count;
    pkv::rope_table_kernel<<<(unsigned)(ctas < most ? ctas : most), 256, 0,
                             static_cast<cudaStream_t>(stream)>>>(p);
    e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

PKV_API pkv_status kv_append_rope(void* k_pool, void* v_pool, const void* k, int64_t k_stride,
                                  const void* v, int64_t v_stride, pkv_dtype dtype,
                                  const int64_t* slot_mapping, const int32_t* positions,
                                  const float* rope_table, int table_positions, int rotary_dim,
                                  int interleaved, const void* q, int64_t q_stride, void* q_out,
                                  int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                  int num_tokens, int n_heads, int n_kv_heads, int head_dim,
                                  int block_size, int num_blocks, void* stream) {
    pkv::AppendRopeParams p;
    std::memset(&p, 0, sizeof(p));
    pkv_status st = fill_append(&p, 2, k_pool, v_pool, k, k_stride, v, v_stride, dtype,
                                slot_mapping, positions, rope_table, table_positions, rotary_dim,
                                interleaved, q, q_stride, q_out, q_out_stride, k_out, k_out_stride,
                                num_tokens, n_heads, n_kv_heads, head_dim, block_size, num_blocks);
    if (st != PKV_OK || num_tokens == 0) return st;
    DeviceInfo* dev = nullptr;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    p.errors = dev->errors;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (head_dim == 128)
        dtype == PKV_BF16 ? launch_append<128, __nv_bfloat16>(p, s) : launch_append<128, __half>(p, s);
    else
        dtype == PKV_BF16 ? launch_append<64, __nv_bfloat16>(p, s) : launch_append<64, __half>(p, s);
    e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

PKV_API pkv_status kv_append_rope_q8(void* k_pool, void* v_pool, float* k_scale, float* v_scale,
                                     const void* k, int64_t k_stride, const void* v,
                                     int64_t v_stride, pkv_dtype dtype,
                                     const int64_t* slot_mapping, const int32_t* positions,
                                     const float* rope_table, int table_positions, int rotary_dim,
                                     int interleaved, const void* q, int64_t q_stride, void* q_out,
                                     int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                     int num_tokens, int n_heads, int n_kv_heads, int head_dim,
                                     int block_size, int num_blocks, void* stream) {
    if (block_size != 16 && block_size != 32) return unsupported("block_size 16 or 32");
    pkv::AppendRopeParams p;
    std::memset(&p, 0, sizeof(p));
    pkv_status st = fill_append(&p, 1, k_pool, v_pool, k, k_stride, v, v_stride, dtype,
                                slot_mapping, positions, rope_table, table_positions, rotary_dim,
                                interleaved, q, q_stride, q_out, q_out_stride, k_out, k_out_stride,
                                num_tokens, n_heads, n_kv_heads, head_dim, block_size, num_blocks);
    if (st != PKV_OK || num_tokens == 0) return st;
    if (num_blocks > 0 && (!k_scale || !v_scale)) return invalid("k_scale or v_scale is NULL");
    if (!aligned4(k_scale) || !aligned4(v_scale)) return invalid("scales must be 4-byte aligned");
    const size_t scales = (size_t)num_blocks * n_kv_heads * sizeof(float);
    if (num_blocks > 0 && pool_span(k_scale, scales).meets(pool_span(v_scale, scales)))
        return invalid("k_scale and v_scale overlap");
    const size_t pool = (size_t)num_blocks * block_size * n_kv_heads * head_dim;
    for (const Span& s : {pool_span(k_scale, scales), pool_span(v_scale, scales)})
        if (num_blocks > 0 &&
            (s.meets(pool_span(k_pool, pool)) || s.meets(pool_span(v_pool, pool))))
            return invalid("the scales overlap a pool");
    DeviceInfo* dev = nullptr;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.errors = dev->errors;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (head_dim == 128)
        dtype == PKV_BF16 ? launch_append_q8<128, __nv_bfloat16>(p, dev->sm_count, s)
                          : launch_append_q8<128, __half>(p, dev->sm_count, s);
    else
        dtype == PKV_BF16 ? launch_append_q8<64, __nv_bfloat16>(p, dev->sm_count, s)
                          : launch_append_q8<64, __half>(p, dev->sm_count, s);
    e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

}  // extern "C"
