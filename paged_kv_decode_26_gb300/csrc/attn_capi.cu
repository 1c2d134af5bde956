// attn_capi.cu -- pkv_attn_prompt of the C ABI: validation, tensor maps, launch.
// Declarations and contracts: pagedkv.h.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "attn_host.h"
#include "attn_prompt_launch.h"
#include "capi_host.h"

using namespace pkv::host;

namespace {

// Prompts of this length and K and V of these bytes (what L2 holds) are worked
// on in bands of items.
constexpr int kBandLength = 4096;
constexpr double kBandBytes = 128e6;

}  // namespace

namespace pkv {
namespace host {

cudaError_t encode_rows_map(CUtensorMap* map, const void* x, pkv_dtype dt, int rows, int heads,
                            int head_dim, long long row_stride, int box_heads, int box_rows) {
    auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t es = 2;
    cuuint64_t dims[4] = {64, (cuuint64_t)head_dim / 64, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[3] = {64 * es, (cuuint64_t)head_dim * es, (cuuint64_t)row_stride * es};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = encode(map, dt == PKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        4, const_cast<void*>(x), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t encode_out_map(CUtensorMap* map, void* out, pkv_dtype dt, int rows, int heads,
                           long long parts, long long head_bytes, long long row_bytes, int group) {
    auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint32_t cols = dt == PKV_F32 ? 32 : 64;
    cuuint64_t dims[4] = {cols, (cuuint64_t)parts, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[3] = {128, (cuuint64_t)head_bytes, (cuuint64_t)row_bytes};
    cuuint32_t box[4] = {cols, 1, (cuuint32_t)group, (cuuint32_t)(32 / group)};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = encode(map,
                        dt == PKV_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                        : dt == PKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        4, out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int attn_stages(int head_dim, int smem_optin) {
    int stages = 8;
    while (stages > 2 && pkv::attn_tc_smem_bytes(head_dim, stages) > (size_t)smem_optin) --stages;
    return stages;
}

}  // namespace host
}  // namespace pkv

extern "C" {

PKV_API pkv_status pkv_attn_prompt(void* out, pkv_dtype out_dtype, const void* q, int64_t q_stride,
                               const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               pkv_dtype dtype, const int32_t* q_start, int num_seqs, int total_q,
                               int max_len, int n_heads, int n_kv_heads, int head_dim, float scale,
                               void* stream) {
    if (num_seqs < 0 || total_q < 0 || max_len < 0) return invalid("sizes");
    if (n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads)
        return invalid("n_heads must be a positive multiple of n_kv_heads");
    if (dtype != PKV_BF16 && dtype != PKV_F16) return unsupported("dtype must be F16 or BF16");
    if (out_dtype != PKV_BF16 && out_dtype != PKV_F16 && out_dtype != PKV_F32)
        return invalid("out_dtype");
    if (!supported_shape(n_heads, n_kv_heads, head_dim, 16))
        return unsupported("head_dim 64/128, group 1/2/4/8");
    if (!std::isfinite(scale)) return invalid("scale is not finite");
    // a larger max_len than there are tokens only adds empty work items
    if (max_len > total_q) max_len = total_q;
    if (max_len > 0x7fffffff - 1024) return unsupported("max_len");
    const int64_t q_row = (int64_t)n_heads * head_dim, kv_row = (int64_t)n_kv_heads * head_dim;
    if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row)
        return invalid("token strides below the rows' elements");
    if (q_stride % 8 || k_stride % 8 || v_stride % 8)
        return invalid("token strides must be multiples of 8 elements");
    if (q_stride >= 1ll << 38 || k_stride >= 1ll << 38 || v_stride >= 1ll << 38)
        return unsupported("token stride");
    if (num_seqs == 0 || total_q == 0 || max_len == 0) return PKV_OK;
    if (!out || !q || !k || !v || !q_start) return invalid("NULL pointer");
    if (!aligned16(out) || !aligned16(q) || !aligned16(k) || !aligned16(v))
        return invalid("out, q, k and v must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(q_start) & 3u) != 0)
        return invalid("q_start must be 4-byte aligned");
    const int G = n_heads / n_kv_heads;
    const int row_tiles = pkv::attn_row_tiles(out_dtype == PKV_F32);
    const int item_tokens = row_tiles * pkv::kAtRows / G;
    const int tiles = (max_len + item_tokens - 1) / item_tokens;
    if ((long long)n_kv_heads * num_seqs > 0x7fffffffLL ||
        (long long)n_kv_heads * ((long long)tiles + 8) > 0x7fffffffLL)
        return unsupported("n_kv_heads * num_seqs or n_kv_heads * max_len too large");
    DeviceInfo* dev = nullptr;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    pkv::AttnLaunch L;
    std::memset(&L, 0, sizeof(L));
    if ((e = encode_rows_map(&L.tm_q, q, dtype, total_q, n_heads, head_dim, q_stride, G,
                             pkv::kAtRows / G)) ||
        (e = encode_rows_map(&L.tm_k, k, dtype, total_q, n_kv_heads, head_dim, k_stride, 1,
                             pkv::kAtKeys)) ||
        (e = encode_rows_map(&L.tm_v, v, dtype, total_q, n_kv_heads, head_dim, v_stride, 1,
                             pkv::kAtKeys)) ||
        (e = encode_out_map(&L.tm_o, out, out_dtype, total_q, n_heads,
                            head_dim * (out_dtype == PKV_F32 ? 4 : 2) / 128,
                            q_row / n_heads * (out_dtype == PKV_F32 ? 4 : 2),
                            q_row * (out_dtype == PKV_F32 ? 4 : 2), G)))
        return cuda_fail(e);
    pkv::AttnParams& p = L.p;
    p.out = out;
    p.out_dtype = out_dtype;
    p.n_heads = n_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = G;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.stages = attn_stages(head_dim, dev->smem_optin);
    p.row_tiles = row_tiles;
    p.tiles = tiles;
    // Items are handed out longest first over all sequences and heads.  Where
    // that would stream K and V from DRAM again for every item (more of them
    // than L2 holds, read by many items each), eight items of a head go
    // together (GB300: prompts of 4096-8192 tokens, 32 heads, 201 MB of K and V,
    // 600 and 575 us, and 650 / 590 back to back, where power limits the clock;
    // 16 of 4096, 8 kv heads, 268 MB, 1524 / 1379; but 16 of 2048, 134 MB, 450 /
    // 467, and 6 of 4096, 101 MB, 595 / 605).
    const double kv_bytes = 4.0 * total_q * n_kv_heads * head_dim;
    p.band = max_len >= kBandLength && kv_bytes >= kBandBytes ? 8 : 1;
    p.total_q = total_q;
    p.max_len = max_len;
    p.v = v;
    p.v_stride = v_stride;
    p.errors = dev->errors;
    L.smem_bytes = pkv::attn_tc_smem_bytes(head_dim, p.stages);
    L.stream = static_cast<cudaStream_t>(stream);
    const bool precise = out_dtype == PKV_F32;
    // one launch, unless the bounds allow 2^31 items
    const long long per_seq = (long long)n_kv_heads * ((tiles + p.band - 1) / p.band * p.band);
    const int step = (int)std::min((long long)num_seqs, 0x7fffffffLL / per_seq);
    for (long long s0 = 0; s0 < num_seqs; s0 += step) {
        p.q_start = q_start + s0;
        p.num_seqs = (int)std::min((long long)step, num_seqs - s0);
        p.n_items = per_seq * p.num_seqs;
        // Where there are more items than SMs, a CTA per item, and running CTAs
        // take over the waiting ones' items, so that the SMs finish together
        // (GB300, taken over and dealt out in turn: prompts of 6.8K and 8K tokens
        // 576 and 721 us, one of 8192 with 4 kv heads 169 and 204; of 128-2048
        // tokens, 8 kv heads, 179 and 171, 64 of 512 204 and 206, 300 of 100 180
        // and 157).  Where most items of the longest sequence's count are empty --
        // lengths that differ much, or a loose max_len -- the CTAs pass over those
        // 32 at a time instead (the 128-2048 under a max_len of 32768: 171, taken
        // over 301), and a long sequence's items may meet few of the CTAs (8192
        // tokens beside 37 of 64: 5.6 ms, taken over 0.23-0.4).
        const long long real =
            (long long)n_kv_heads * ((long long)total_q / item_tokens + p.num_seqs);
        p.dynamic = p.n_items > dev->sm_count && p.n_items <= 2 * real;
        L.ctas = (int)(p.dynamic || p.n_items < dev->sm_count ? p.n_items : dev->sm_count);
        e = dtype == PKV_BF16 ? pkv::launch_attn_prompt_bf16(head_dim, precise, L)
                              : pkv::launch_attn_prompt_f16(head_dim, precise, L);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return PKV_OK;
}

}  // extern "C"
