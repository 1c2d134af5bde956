// q8_capi.cu -- the C ABI's attention over 8-bit pages (paged_attn_decode_q8,
// paged_attn_multi_query_q8): validation, workspace layout and launches.
// Declarations and contracts: pagedkv.h.
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "capi_host.h"
#include "decode_launch.h"
#include "decode_q8_launch.h"
#include "multi_query_q8_launch.h"
#include "pieces_host.h"

using namespace pkv::host;

namespace {

// The pool [num_blocks, B, Hk, D] of bytes as a 4-D tensor: dims (D, B, Hk,
// blocks), box (D, 16, 1, 1), swizzled over D bytes: one load brings 16 tokens of
// one kv head as [16][D].
cudaError_t encode_q8_map(CUtensorMap* map, const void* pool, int num_blocks, int block_size,
                          int n_kv_heads, int head_dim) {
    auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t D = (cuuint64_t)head_dim, row = D * n_kv_heads;
    cuuint64_t dims[4] = {D, (cuuint64_t)block_size, (cuuint64_t)n_kv_heads,
                          (cuuint64_t)num_blocks};
    cuuint64_t strides[3] = {row, D, (cuuint64_t)block_size * row};
    cuuint32_t box[4] = {(cuuint32_t)head_dim, 16, 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(pool), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Without blocks nothing is loaded; the maps need some valid tensor: q.
cudaError_t encode_q8_maps(pkv::Q8Launch* L, const void* k_pool, const void* v_pool, const void* q,
                           int num_blocks, int block_size, int n_kv_heads, int head_dim) {
    const int n = num_blocks > 0 ? num_blocks : 1;
    const cudaError_t e = encode_q8_map(&L->tm_k, num_blocks > 0 ? k_pool : q, n, block_size,
                                        n_kv_heads, head_dim);
    return e != cudaSuccess ? e
                            : encode_q8_map(&L->tm_v, num_blocks > 0 ? v_pool : q, n, block_size,
                                            n_kv_heads, head_dim);
}

// Contexts up to kShortContext tokens are decoded whole, by a CTA per kv head
// (decode_q8_short_kernel), where there are at most kShortPairs of them per SM.
// GB300, whole / in pieces, us: 64 pairs of 64 tokens 5.1 / 16.1, of 512 10.5 / 16.2,
// of 1024 16.6 / 17.4, of 2048 29 / 18; 1024 pairs of up to 256 17 / 23, of up to
// 1024 38 / 40, of up to 2048 69 / 58; 2048 pairs of up to 64 22.8 / 22.4, of up to
// 512 46 / 40.
// Warps of such a CTA: kQ8ShortWarps where every SM has one at most, else 4.  4 / 12
// warps: 32 pairs of up to 200 tokens 5.8 / 4.6, 128 of 512 9.4 / 7.0, of 1024 15.8 /
// 9.4; 1024 of up to 256 24 / 39.
constexpr int kShortContext = 1024;
constexpr int kShortPairs = 7;
// Warps per context, 0: not whole.
int whole_contexts(long long pairs, int max_context_len, int sm_count) {
    if (max_context_len > kShortContext || pairs > (long long)kShortPairs * sm_count) return 0;
    return pairs <= sm_count ? pkv::kQ8ShortWarps : 4;
}

constexpr PiecesKind kPiecesQ8 = {pkv::kQ8Tokens, pkv::kQ8Warps, pkv::kQ8StreamHeads};

PiecesGrid q8_grid(int num_seqs, int n_kv_heads, int max_context_len, int sm_count) {
    return pieces_grid(num_seqs, n_kv_heads, max_context_len, sm_count, false, kPiecesQ8);
}

pkv_status check_scales(const float* k_scale, const float* v_scale, int num_blocks) {
    if (num_blocks > 0 && (!k_scale || !v_scale)) return invalid("k_scale or v_scale is NULL");
    if (!aligned4(k_scale) || !aligned4(v_scale)) return invalid("scales must be 4-byte aligned");
    return PKV_OK;
}

// The output is the queries themselves (every row is read by those that write it, before
// they do) or lies apart from all that is read.
pkv_status check_apart(const void* out, pkv_dtype out_dtype, const void* q, size_t elements,
                       const void* k_pool, const void* v_pool, size_t pool, const float* k_scale,
                       const float* v_scale, size_t scales) {
    auto meets = [&](const void* p, size_t bytes) {
        const uintptr_t o = reinterpret_cast<uintptr_t>(out), a = reinterpret_cast<uintptr_t>(p);
        return o < a + bytes && a < o + elements * (out_dtype == PKV_F32 ? 4 : 2);
    };
    if (meets(q, elements * 2) && (out != q || out_dtype == PKV_F32))
        return invalid("out overlaps q (it may be q itself, in 16 bits)");
    if (meets(k_pool, pool) || meets(v_pool, pool) || meets(k_scale, scales * sizeof(float)) ||
        meets(v_scale, scales * sizeof(float)))
        return invalid("out overlaps the cache");
    return PKV_OK;
}

// How a chunk's items (pairs of row tiles of a kv head) meet the SMs, one at a time on
// each.  Items that do not fill the SMs once more (all of them, where there are fewer
// than SMs) are cut into parts of their keys, kPartTiles key tiles at least, so that the
// last round is short: as many as make it shortest, at kItemTiles key tiles for a
// part's start and end and kMergeTiles for the launch that merges.  GB300, us, whole / in
// parts: 2 chunks of 2048 tokens behind 12K-16K, 32 heads 904 / 840; of 1500 tokens at
// 4000, 32 query and 8 kv heads, 117 / 103, of 100 at 8192 120 / 35; 2 chunks of 2 tokens, 4
// heads, at 16000 229 / 27; 16 of up to 8 tokens at up to 1000, 16 query and 4 kv heads 16.6
// / 16.1; of 512 tokens at 600 23.1 / 27.8, therefore whole.
// A few tokens with short contexts go to the decode of whole contexts, 8 / G tokens to a
// CTA, where its CTAs are all on the SMs at once (their rings: two a SM at head_dim 64, one
// at 128).  Row tiles / so, us, head_dim 64, 16 query and 4 kv heads: 16 sequences of 8
// tokens at 900-1000 18.8 / 14.1, of up to 8 at up to 1000 16.1 / 11.2, 1 of 2 tokens 13.9
// / 10.0, of 150 21.3 / 14.1; head_dim 128, 32 and 8 heads, 4 of up to 16 at 900 (256
// CTAs) 17.7 / 23.9.
constexpr int kPartTiles = 4;
constexpr int kItemTiles = 2;
constexpr int kMergeTiles = 3;
struct ChunkShape {
    int tiles;            // pairs of row tiles of the longest chunk allowed
    long long items;
    long long whole;      // items that are not cut
    int splits;           // parts of the others
    size_t o, ml, heads, end;    // workspace
    int by_token;         // warps of a CTA that decodes whole contexts, 0: row tiles
};
ChunkShape chunk_shape(int num_seqs, int max_q_len, int n_heads, int n_kv_heads, int head_dim,
                       int max_context_len, int sm_count) {
    ChunkShape c;
    std::memset(&c, 0, sizeof(c));
    const int G = n_heads / n_kv_heads, cta_tokens = 2 * pkv::kMq8Rows / G;
    const long long pairs =
        (long long)num_seqs * n_kv_heads * (((long long)max_q_len + 8 / G - 1) / (8 / G));
    if (pairs <= (long long)sm_count * (128 / head_dim))
        c.by_token = whole_contexts(pairs, max_context_len, sm_count) ? pkv::kQ8ShortWarps : 0;
    if (c.by_token) return c;
    c.tiles = (int)(((long long)max_q_len + cta_tokens - 1) / cta_tokens);
    c.items = (long long)c.tiles * n_kv_heads * num_seqs;
    c.whole = c.items / sm_count * sm_count;
    c.splits = 1;
    const long long others = c.items - c.whole;
    const long long key_tiles = ((long long)max_context_len + pkv::kMq8Keys - 1) / pkv::kMq8Keys;
    long long best = key_tiles + kItemTiles;
    for (int k = 2; others > 0 && k <= sm_count && k * kPartTiles <= key_tiles; ++k) {
        const long long rounds = (others * k + sm_count - 1) / sm_count;
        const long long time = rounds * ((key_tiles + k - 1) / k + kItemTiles) + kMergeTiles;
        if (time < best) {
            best = time;
            c.splits = k;
        }
    }
    if (c.splits == 1) {
        c.whole = c.items;
        return c;
    }
    const size_t rows = (size_t)others * c.splits * 2 * pkv::kMq8Rows;
    c.ml = align256(rows * head_dim * sizeof(float));
    c.heads = align256(c.ml + rows * 2 * sizeof(float));
    c.end = align256(c.heads + (size_t)others * sizeof(int4));
    return c;
}

// Longest context first (longest_first): the items that end last begin first, but every
// CTA ranks the sequences, and neighbours no longer share a head's keys.  In order /
// longest first, us, chunks of 8 to 8192 / S tokens, 32 query and 8 kv heads: 8 sequences
// at 1000-8000 183 / 152, 1000-3000 95 / 92, 64-500 43 / 41; 32 at 500-3000 192 / 187,
// 256-2500 156 / 162; 64 at 500-4000 260 / 233, 64-500 97 / 99; 128 at 1000-8000 580 / 544,
// 256-2000 206 / 211; 256 at 1000-16000 1949 / 1920, 500-4000 602 / 628.  Prompts (chunks
// that are most of their contexts), 4 of 500-8000 1090 / 1067, 16 of 100-4000 924 / 932, 64
// of 20-3000 2200 / 2357.  2 equal chunks of 2048 at 12K-16K 739 / 709, 32 / 32 heads 693 /
// 721.
constexpr int kLptMaxSeqs = 256;
constexpr int kLptMinContext = 2560, kLptSeqContext = 32, kLptPromptContext = 8192;
bool longest_first_pays(int num_seqs, int max_q_len, int max_context_len) {
    const int from = max_q_len > max_context_len / 2
                         ? kLptPromptContext
                         : std::max(kLptMinContext, kLptSeqContext * num_seqs);
    return num_seqs <= kLptMaxSeqs && max_context_len >= from;
}

}  // namespace

extern "C" {

PKV_API size_t pkv_decode_q8_workspace_bytes(int num_seqs, int n_heads, int n_kv_heads,
                                             int head_dim, int block_size, int max_context_len) {
    if (!supported_shape(n_heads, n_kv_heads, head_dim, block_size) || num_seqs <= 0 ||
        max_context_len < 0)
        return 0;
    DeviceInfo* dev = nullptr;
    const int sms = device_info(&dev) == cudaSuccess ? dev->sm_count : kDefaultSms;
    if (whole_contexts((long long)num_seqs * n_kv_heads, max_context_len, sms)) return 0;
    return pieces_workspace(num_seqs, n_heads, n_kv_heads, head_dim,
                            q8_grid(num_seqs, n_kv_heads, max_context_len, sms))
        .end;
}

PKV_API pkv_status paged_attn_decode_q8(
    void* out, pkv_dtype out_dtype, const void* q, pkv_dtype q_dtype, const void* k_pool,
    const void* v_pool, const float* k_scale, const float* v_scale, const int32_t* block_tables,
    int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int n_heads,
    int n_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
    int max_context_len, void* workspace, size_t workspace_bytes, void* stream) {
    pkv_status st = check_paged_decode(out, out_dtype, q, k_pool, v_pool, q_dtype, block_tables,
                                       max_blocks_per_seq, context_lens, num_seqs, n_heads,
                                       n_kv_heads, head_dim, block_size, num_blocks, scale,
                                       max_context_len);
    if (st != PKV_OK || num_seqs == 0) return st;
    if ((st = check_scales(k_scale, v_scale, num_blocks)) != PKV_OK) return st;
    const size_t scales = (size_t)num_blocks * n_kv_heads;
    if ((st = check_apart(out, out_dtype, q, (size_t)num_seqs * n_heads * head_dim, k_pool, v_pool,
                          scales * block_size * head_dim, k_scale, v_scale, scales)) != PKV_OK)
        return st;
    DeviceInfo* dev = nullptr;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const PiecesGrid pieces = q8_grid(num_seqs, n_kv_heads, max_context_len, dev->sm_count);
    const PiecesWorkspace w =
        pieces_workspace(num_seqs, n_heads, n_kv_heads, head_dim, pieces);
    pkv::Q8Launch L;
    std::memset(&L, 0, sizeof(L));
    L.whole = whole_contexts((long long)num_seqs * n_kv_heads, max_context_len, dev->sm_count);
    if (!L.whole && (st = check_workspace(workspace, workspace_bytes, w.end)) != PKV_OK) return st;
    L.stream = static_cast<cudaStream_t>(stream);
    if ((e = encode_q8_maps(&L, k_pool, v_pool, q, num_blocks, block_size, n_kv_heads,
                            head_dim)) != cudaSuccess)
        return cuda_fail(e);
    pkv::Q8Params& p = L.p;
    fill_piece_problem(&p, pieces, out, out_dtype, q, block_tables, max_blocks_per_seq,
                       context_lens, num_seqs, n_heads, n_kv_heads, block_size, num_blocks, scale,
                       max_context_len, w, workspace, *dev);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    e = q_dtype == PKV_BF16 ? pkv::launch_decode_q8_bf16(head_dim, L)
                            : pkv::launch_decode_q8_f16(head_dim, L);
    if (e != cudaSuccess) return cuda_fail(e);
    if (L.whole) return PKV_OK;
    // (pieces of a row to expect, and warps that merge them: as the shared decode)
    const long long streams =
        (long long)p.ctas * (pkv::kQ8Warps / p.stream_heads);
    const long long pairs = (long long)num_seqs * (n_kv_heads / p.stream_heads);
    const bool few = 2 + streams / pairs <= 12;
    const int rows = few ? pkv::kFinishWarps : 1;
    const dim3 grid((unsigned)((n_heads + rows - 1) / rows), (unsigned)num_seqs);
    auto merge = head_dim == 128
                     ? (few ? pkv::decode_q8_finish_kernel<128, 1> : pkv::decode_q8_finish_kernel<128, 4>)
                     : (few ? pkv::decode_q8_finish_kernel<64, 1> : pkv::decode_q8_finish_kernel<64, 4>);
    e = launch_dependent(merge, grid, pkv::kFinishThreads, 0, L.stream,
                         static_cast<const pkv::PieceParams&>(p));
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

PKV_API size_t pkv_multi_query_q8_workspace_bytes(int num_seqs, int max_q_len, int n_heads,
                                                  int n_kv_heads, int head_dim, int block_size,
                                                  int max_context_len) {
    if (!supported_shape(n_heads, n_kv_heads, head_dim, block_size) || num_seqs <= 0 ||
        max_q_len <= 0 || max_context_len < 0)
        return 0;
    DeviceInfo* dev = nullptr;
    const int sms = device_info(&dev) == cudaSuccess ? dev->sm_count : kDefaultSms;
    return chunk_shape(num_seqs, max_q_len, n_heads, n_kv_heads, head_dim, max_context_len, sms).end;
}

PKV_API pkv_status paged_attn_multi_query_q8(
    void* out, pkv_dtype out_dtype, const void* q, pkv_dtype q_dtype, const int32_t* q_start,
    int total_q, int max_q_len, const void* k_pool, const void* v_pool, const float* k_scale,
    const float* v_scale, const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int num_seqs, int n_heads, int n_kv_heads, int head_dim,
    int block_size, int num_blocks, float scale, int max_context_len, void* workspace,
    size_t workspace_bytes, void* stream) {
    if (total_q < 0 || max_q_len < 0) return invalid("sizes");
    const bool none = num_seqs == 0 || total_q == 0 || max_q_len == 0;
    pkv_status st = check_paged_decode(out, out_dtype, q, k_pool, v_pool, q_dtype, block_tables,
                                       max_blocks_per_seq, context_lens, none ? 0 : num_seqs,
                                       n_heads, n_kv_heads, head_dim, block_size, num_blocks,
                                       scale, max_context_len);
    if (st != PKV_OK) return st;
    if (num_seqs < 0) return invalid("sizes");
    if (none) return PKV_OK;
    if (!q_start) return invalid("q_start is NULL");
    if (!aligned4(q_start)) return invalid("q_start must be 4-byte aligned");
    if ((st = check_scales(k_scale, v_scale, num_blocks)) != PKV_OK) return st;
    const size_t scales = (size_t)num_blocks * n_kv_heads;
    if ((st = check_apart(out, out_dtype, q, (size_t)total_q * n_heads * head_dim, k_pool, v_pool,
                          scales * block_size * head_dim, k_scale, v_scale, scales)) != PKV_OK)
        return st;
    DeviceInfo* dev = nullptr;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    ChunkShape c = chunk_shape(num_seqs, max_q_len, n_heads, n_kv_heads, head_dim,
                               max_context_len, dev->sm_count);
    // (shorter chunks than the longest: how many items there are is not known here)
    if (c.whole > 0 && total_q != (long long)num_seqs * max_q_len) {
        c.whole = c.items;
        c.splits = 1;
    }
    if (!c.by_token && c.whole + (c.items - c.whole) * c.splits > INT_MAX) return invalid("sizes");
    if (c.splits > 1 && (st = check_workspace(workspace, workspace_bytes, c.end)) != PKV_OK)
        return st;
    if (c.by_token) {
        pkv::Q8Launch L;
        std::memset(&L, 0, sizeof(L));
        L.whole = c.by_token;
        L.stream = static_cast<cudaStream_t>(stream);
        if ((e = encode_q8_maps(&L, k_pool, v_pool, q, num_blocks, block_size, n_kv_heads,
                                head_dim)) != cudaSuccess)
            return cuda_fail(e);
        pkv::Q8Params& p = L.p;
        PiecesWorkspace w;
        std::memset(&w, 0, sizeof(w));
        const int blocks = (max_context_len + block_size - 1) / block_size;
        fill_piece_problem(&p, q8_grid(num_seqs, n_kv_heads, max_context_len, dev->sm_count), out,
                           out_dtype, q, block_tables, max_blocks_per_seq, context_lens, num_seqs,
                           n_heads, n_kv_heads, block_size, num_blocks, scale, blocks * block_size,
                           w, nullptr, *dev);
        p.k_scale = k_scale;
        p.v_scale = v_scale;
        p.q_start = q_start;
        p.total_q = total_q;
        p.max_q_len = max_q_len;
        p.v_codes = static_cast<const unsigned char*>(v_pool);
        e = q_dtype == PKV_BF16 ? pkv::launch_decode_q8_bf16(head_dim, L)
                                : pkv::launch_decode_q8_f16(head_dim, L);
        return e == cudaSuccess ? PKV_OK : cuda_fail(e);
    }
    pkv::Mq8Launch L;
    std::memset(&L, 0, sizeof(L));
    pkv::Mq8Params& p = L.p;
    p.out = out;
    p.out_dtype = out_dtype;
    p.q = q;
    p.q_bf16 = q_dtype == PKV_BF16;
    p.q_start = q_start;
    p.total_q = total_q;
    p.max_q_len = max_q_len;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.num_seqs = num_seqs;
    p.n_heads = n_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = n_heads / n_kv_heads;
    p.num_blocks = num_blocks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.max_pages = (int)(((long long)max_context_len + block_size - 1) / block_size);
    p.errors = dev->errors;
    p.lpt_seqs = longest_first_pays(num_seqs, max_q_len, max_context_len) ? num_seqs : 0;
    p.tiles = c.tiles;
    p.whole = (int)c.whole;
    p.splits = c.splits;
    p.block_size = block_size;
    if (c.splits > 1) {
        unsigned char* ws = static_cast<unsigned char*>(workspace);
        p.part_o = reinterpret_cast<float*>(ws + c.o);
        p.part_ml = reinterpret_cast<float*>(ws + c.ml);
        p.heads = reinterpret_cast<int4*>(ws + c.heads);
    }
    const long long others = c.items - c.whole;
    L.ctas = (unsigned)(c.whole + others * c.splits);
    L.stream = static_cast<cudaStream_t>(stream);
    e = pkv::launch_multi_query_q8(head_dim, block_size, L);
    if (e == cudaSuccess && c.splits > 1) {
        const long long rows = std::min(2LL * pkv::kMq8Rows, (long long)max_q_len * p.group);
        const dim3 grid((unsigned)others,
                        (unsigned)((rows + pkv::kMq8MergeRows - 1) / pkv::kMq8MergeRows));
        e = launch_dependent(head_dim == 128 ? pkv::multi_query_q8_merge_kernel<128>
                                             : pkv::multi_query_q8_merge_kernel<64>,
                             grid, pkv::kMq8MergeThreads, 0, L.stream, p);
    }
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

}  // extern "C"
