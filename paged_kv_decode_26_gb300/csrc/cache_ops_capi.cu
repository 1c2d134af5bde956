// cache_ops_capi.cu -- the C ABI's cache-budget calls: the decode that
// accumulates attention weights (paged_attn_decode_weights) and the eviction
// that goes by them (kv_evict): validation, workspace layout and launches.
// Declarations and contracts: pagedkv.h.
#include <cudaTypedefs.h>

#include <cmath>
#include <cstring>

#include "capi_host.h"
#include "decode_launch.h"
#include "decode_weights_launch.h"
#include "evict_kernels.cuh"
#include "pieces_host.h"

using namespace pkv::host;

namespace {

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

}  // namespace

namespace pkv {
namespace host {

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

int pieces_stream_heads(int n_kv_heads) {
    int hw = kPieceWarps;
    while (n_kv_heads % hw) hw /= 2;
    return hw;
}

PiecesGrid pieces_grid(int num_seqs, int n_kv_heads, int max_context_len, int sm_count,
                       bool short_runs) {
    const int hw = pieces_stream_heads(n_kv_heads), per_cta = kPieceWarps / hw;
    const long long chunks = (long long)num_seqs * (n_kv_heads / hw) *
                             (((long long)max_context_len + kPieceTokens - 1) / kPieceTokens);
    const long long streams = (chunks + kPieceMinRun - 1) / kPieceMinRun;
    const long long ctas = (streams + per_cta - 1) / per_cta;
    PiecesGrid g;
    g.ctas = (int)(ctas < 1 ? 1 : (ctas < sm_count ? ctas : sm_count));
    g.extra = short_runs && chunks >= (long long)g.ctas * per_cta * kPieceDealt
                  ? kPieceExtra * g.ctas
                  : 0;
    return g;
}

PiecesWorkspace pieces_workspace(int num_seqs, int n_heads, int n_kv_heads, int head_dim,
                                 const PiecesGrid& grid) {
    PiecesWorkspace w;
    const size_t rows = (size_t)num_seqs * n_heads + (size_t)(grid.ctas + grid.extra) *
                                                         kPieceWarps * (n_heads / n_kv_heads);
    const size_t pairs = (size_t)num_seqs * n_kv_heads;
    w.o = 0;
    w.ml = align256(w.o + rows * head_dim * sizeof(float));
    w.seg_first = align256(w.ml + rows * 2 * sizeof(float));
    w.seg_last = align256(w.seg_first + pairs * sizeof(int));
    w.end = align256(w.seg_last + pairs * sizeof(int));
    return w;
}

pkv_status check_paged_decode(const void* out, pkv_dtype out_dtype, const void* q,
                              const void* k_pool, const void* v_pool, pkv_dtype kv_dtype,
                              const int32_t* block_tables, int max_blocks_per_seq,
                              const int32_t* context_lens, int num_seqs, int n_heads,
                              int n_kv_heads, int head_dim, int block_size, int num_blocks,
                              float scale, int max_context_len) {
    if (num_seqs < 0 || max_context_len < 0) return invalid("sizes");
    if (num_seqs > 65535) return unsupported("more than 65535 sequences per call");
    if (n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads)
        return invalid("n_heads must be a positive multiple of n_kv_heads");
    if (kv_dtype != PKV_BF16 && kv_dtype != PKV_F16)
        return unsupported("kv_dtype must be F16 or BF16");
    if (out_dtype != PKV_BF16 && out_dtype != PKV_F16 && out_dtype != PKV_F32)
        return invalid("out_dtype");
    if (!supported_shape(n_heads, n_kv_heads, head_dim, block_size))
        return unsupported("head_dim 64/128, block_size 16/32, group 1/2/4/8");
    if (n_heads > 4096) return unsupported("more than 4096 query heads");
    if (num_blocks < 0 || max_blocks_per_seq <= 0) return invalid("pool / table sizes");
    if (!table_tokens_fit(max_blocks_per_seq, block_size))
        return unsupported("max_blocks_per_seq * block_size exceeds 2^31 - 1 tokens");
    if (!std::isfinite(scale)) return invalid("scale is not finite");
    if (max_context_len > 0x7fffffff - 1024) return unsupported("max_context_len");
    if ((long long)num_seqs * (((long long)max_context_len + 15) / 16) > 0x7fffffffLL)
        return unsupported("num_seqs * max_context_len exceeds 2^35 tokens");
    if (num_seqs == 0) return PKV_OK;
    if (!out || !q || !block_tables || !context_lens) return invalid("NULL pointer");
    if (num_blocks > 0 && (!k_pool || !v_pool)) return invalid("k_pool or v_pool is NULL");
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool))
        return invalid("out, q, k_pool and v_pool must be 16-byte aligned");
    if (!aligned4(block_tables) || !aligned4(context_lens))
        return invalid("block_tables and context_lens must be 4-byte aligned");
    return PKV_OK;
}

// The pool [num_blocks, B, Hk, D] as a 4-D tensor for the piece decode: dims
// (64, B, Hk D / 64, blocks), box (64, 16, D / 64, 1), 128-byte swizzle: one
// load brings 16 tokens of one kv head as [D / 64][16][64].
static cudaError_t encode_chunk_map(CUtensorMap* map, const void* pool, pkv_dtype dt,
                                    int num_blocks, int block_size, int n_kv_heads,
                                    int head_dim) {
    auto encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t es = 2, row = (cuuint64_t)n_kv_heads * head_dim;
    cuuint64_t dims[4] = {64, (cuuint64_t)block_size, row / 64, (cuuint64_t)num_blocks};
    cuuint64_t strides[3] = {row * es, 64 * es, (cuuint64_t)block_size * row * es};
    cuuint32_t box[4] = {64, (cuuint32_t)kPieceTokens, (cuuint32_t)(head_dim / 64), 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = encode(map, dt == PKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        4, const_cast<void*>(pool), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

pkv_status fill_pieces(PieceParams* pp, CUtensorMap* tm_k, CUtensorMap* tm_v,
                       const PiecesGrid& grid, void* out,
                       pkv_dtype out_dtype, const void* q, const void* k_pool, const void* v_pool,
                       pkv_dtype kv_dtype, const int32_t* block_tables, int max_blocks_per_seq,
                       const int32_t* context_lens, int num_seqs, int n_heads, int n_kv_heads,
                       int head_dim, int block_size, int num_blocks, float scale,
                       int max_context_len, const PiecesWorkspace& w, void* workspace,
                       const DeviceInfo& dev) {
    const int map_blocks = num_blocks > 0 ? num_blocks : 1;
    cudaError_t e;
    if ((e = encode_chunk_map(tm_k, num_blocks > 0 ? k_pool : q, kv_dtype, map_blocks, block_size,
                              n_kv_heads, head_dim)) ||
        (e = encode_chunk_map(tm_v, num_blocks > 0 ? v_pool : q, kv_dtype, map_blocks, block_size,
                              n_kv_heads, head_dim)))
        return cuda_fail(e);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    PieceParams& p = *pp;
    p.out = out;
    p.out_dtype = out_dtype;
    p.q = q;
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.num_seqs = num_seqs;
    p.n_heads = n_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = n_heads / n_kv_heads;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    const long long table = (long long)max_blocks_per_seq * block_size;
    p.cap_tokens = (int)(table < max_context_len ? table : max_context_len);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.stream_heads = pieces_stream_heads(n_kv_heads);
    p.ctas = grid.ctas;
    p.extra_ctas = grid.extra;
    p.ws_o = reinterpret_cast<float*>(ws + w.o);
    p.ws_ml = reinterpret_cast<float*>(ws + w.ml);
    p.seg_first = reinterpret_cast<int*>(ws + w.seg_first);
    p.seg_last = reinterpret_cast<int*>(ws + w.seg_last);
    p.errors = dev.errors;
    return PKV_OK;
}

pkv_status check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (!workspace || bytes < need) {
        invalid("workspace smaller than the call's workspace_bytes()");
        return PKV_ERR_WORKSPACE;
    }
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return invalid("workspace must be 256-byte aligned");
    return PKV_OK;
}

}  // namespace host
}  // namespace pkv

namespace {

// Scores of every head: rows of whole chunks.
size_t score_row(int max_context_len) { return ((size_t)max_context_len + 15) / 16 * 16; }

size_t weights_bytes(int num_seqs, int n_heads, int n_kv_heads, int head_dim, int max_context_len,
                     int sm_count, PiecesWorkspace* w) {
    *w = pieces_workspace(num_seqs, n_heads, n_kv_heads, head_dim,
                          pieces_grid(num_seqs, n_kv_heads, max_context_len, sm_count, true));
    return w->end + align256((size_t)num_seqs * n_heads * score_row(max_context_len) *
                             sizeof(float));
}

}  // namespace

extern "C" {

PKV_API size_t pkv_decode_weights_workspace_bytes(int num_seqs, int n_heads, int n_kv_heads,
                                                  int head_dim, int block_size,
                                                  int max_context_len) {
    if (!supported_shape(n_heads, n_kv_heads, head_dim, block_size) || num_seqs <= 0 ||
        max_context_len < 0)
        return 0;
    DeviceInfo* dev = nullptr;
    const int sms = device_info(&dev) == cudaSuccess ? dev->sm_count : kDefaultSms;
    PiecesWorkspace w;
    return weights_bytes(num_seqs, n_heads, n_kv_heads, head_dim, max_context_len, sms, &w);
}

PKV_API pkv_status paged_attn_decode_weights(
    void* out, pkv_dtype out_dtype, const void* q, const void* k_pool, const void* v_pool,
    pkv_dtype kv_dtype, const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, float* weights, int64_t weight_stride, int num_seqs, int n_heads,
    int n_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
    int max_context_len, void* workspace, size_t workspace_bytes, void* stream) {
    pkv_status st = check_paged_decode(out, out_dtype, q, k_pool, v_pool, kv_dtype, block_tables,
                                       max_blocks_per_seq, context_lens, num_seqs, n_heads,
                                       n_kv_heads, head_dim, block_size, num_blocks, scale,
                                       max_context_len);
    if (st != PKV_OK) return st;
    if (weight_stride < max_context_len) return invalid("weight_stride below max_context_len");
    if (num_seqs == 0) return PKV_OK;
    if (!weights && max_context_len > 0) return invalid("weights is NULL");
    if (!aligned4(weights)) return invalid("weights must be 4-byte aligned");
    DeviceInfo* dev = nullptr;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    PiecesWorkspace w;
    const size_t need = weights_bytes(num_seqs, n_heads, n_kv_heads, head_dim, max_context_len,
                                      dev->sm_count, &w);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != PKV_OK) return st;
    pkv::PiecesLaunch L;
    std::memset(&L, 0, sizeof(L));
    const PiecesGrid pieces =
        pieces_grid(num_seqs, n_kv_heads, max_context_len, dev->sm_count, true);
    L.stream = static_cast<cudaStream_t>(stream);
    pkv::PieceParams& p = L.p;
    st = fill_pieces(&p, &L.tm_k, &L.tm_v, pieces, out, out_dtype, q, k_pool, v_pool, kv_dtype,
                     block_tables, max_blocks_per_seq, context_lens, num_seqs, n_heads,
                     n_kv_heads, head_dim, block_size, num_blocks, scale, max_context_len, w,
                     workspace, *dev);
    if (st != PKV_OK) return st;
    p.scores = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + w.end);
    p.score_stride = (long long)score_row(max_context_len);
    p.weights = weights;
    p.weight_stride = weight_stride;
    e = kv_dtype == PKV_BF16 ? pkv::launch_weights_bf16(head_dim, L)
                             : pkv::launch_weights_f16(head_dim, L);
    if (e != cudaSuccess) return cuda_fail(e);
    const int tiles = (p.cap_tokens + pkv::kWeightTokens - 1) / pkv::kWeightTokens;
    const dim3 grid((unsigned)(n_heads + tiles), (unsigned)num_seqs);
    const size_t merge = (size_t)pkv::kFinishWarps * head_dim * sizeof(float);
    const size_t sums = (size_t)n_heads * sizeof(float2);
    const size_t smem = merge > sums ? merge : sums;
    e = head_dim == 128
            ? launch_dependent(pkv::decode_weights_finish_kernel<128>, grid, pkv::kFinishThreads,
                               smem, L.stream, p)
            : launch_dependent(pkv::decode_weights_finish_kernel<64>, grid, pkv::kFinishThreads,
                               smem, L.stream, p);
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

PKV_API pkv_status kv_evict(void* k_pool, void* v_pool, pkv_dtype dtype,
                            const int32_t* block_tables, int max_blocks_per_seq,
                            const int32_t* context_lens, const float* weights,
                            int64_t weight_stride, int weight_cols, const int32_t* new_tables,
                            int new_blocks_per_seq, int32_t* new_lens, float* new_weights,
                            int64_t new_weight_stride, int new_weight_cols, int32_t* kept,
                            int num_seqs, int keep, int recent, int n_kv_heads, int head_dim,
                            int block_size, int num_blocks, void* stream) {
    if (num_seqs < 0 || n_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks < 0 ||
        max_blocks_per_seq <= 0 || new_blocks_per_seq <= 0 || weight_cols < 0)
        return invalid("sizes");
    if (num_seqs > 65535) return unsupported("more than 65535 sequences per call");
    if (keep < 1 || recent < 0 || recent > keep)
        return invalid("keep >= 1 and 0 <= recent <= keep");
    if (!table_tokens_fit(max_blocks_per_seq, block_size))
        return unsupported("max_blocks_per_seq * block_size exceeds 2^31 - 1 tokens");
    if ((long long)new_blocks_per_seq * block_size < keep)
        return invalid("new_tables cannot hold keep tokens");
    if (weight_stride < weight_cols || new_weight_stride < new_weight_cols ||
        new_weight_cols < keep)
        return invalid("weight rows: strides below the columns, or new_weights below keep columns");
    const long long table = (long long)max_blocks_per_seq * block_size;
    const long long cap_tokens = table < weight_cols ? table : weight_cols;
    if (cap_tokens > pkv::kEvictMost || new_weight_cols > pkv::kEvictMost)   // (keep is below)
        return unsupported("contexts or new_weight_cols above 2^31 - 2^14");
    int es = 0;
    switch (dtype) {
        case PKV_F16:
        case PKV_BF16: es = 2; break;
        case PKV_F32: es = 4; break;
        default: return invalid("dtype");
    }
    const long long row_bytes = (long long)n_kv_heads * head_dim * es;
    if (row_bytes % 16)
        return unsupported("n_kv_heads * head_dim * element size must be a multiple of 16 bytes");
    if (row_bytes / 16 > 0x7fffffffLL) return unsupported("row too large");
    if (num_seqs == 0) return PKV_OK;
    if (!block_tables || !context_lens || !weights || !new_tables || !new_lens || !new_weights ||
        !kept)
        return invalid("NULL pointer");
    if (num_blocks > 0 && (!k_pool || !v_pool)) return invalid("k_pool or v_pool is NULL");
    if (!aligned16(k_pool) || !aligned16(v_pool)) return invalid("pools must be 16-byte aligned");
    for (const void* x : {(const void*)block_tables, (const void*)context_lens,
                          (const void*)weights, (const void*)new_tables, (const void*)new_lens,
                          (const void*)new_weights, (const void*)kept})
        if (!aligned4(x)) return invalid("tables, lengths, weights and kept must be 4-byte aligned");
    // the second kernel reads what the first one read: outputs may not lie on inputs
    const size_t n = (size_t)num_seqs;
    const struct {
        const void* p;
        size_t bytes;
    } in[] = {{block_tables, n * max_blocks_per_seq * 4},
              {context_lens, n * 4},
              {weights, ((n - 1) * (size_t)weight_stride + (size_t)weight_cols) * 4},
              {new_tables, n * new_blocks_per_seq * 4}},
      outs[] = {{new_lens, n * 4},
                {new_weights, ((n - 1) * (size_t)new_weight_stride + (size_t)new_weight_cols) * 4},
                {kept, n * (size_t)keep * 4}};
    for (const auto& o : outs) {
        for (const auto& i : in)
            if (overlap(o.p, o.bytes, i.p, i.bytes))
                return invalid("new_lens, new_weights and kept may not overlap the inputs");
        for (const auto& i : outs)
            if (i.p != o.p && overlap(o.p, o.bytes, i.p, i.bytes))
                return invalid("new_lens, new_weights and kept may not overlap");
    }
    if (outs[0].p == outs[1].p || outs[1].p == outs[2].p || outs[0].p == outs[2].p)
        return invalid("new_lens, new_weights and kept may not overlap");
    DeviceInfo* dev = nullptr;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return cuda_fail(e);

    pkv::EvictParams p;
    std::memset(&p, 0, sizeof(p));
    p.block_tables = block_tables;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.weights = weights;
    p.weight_stride = weight_stride;
    p.cap_tokens = (int)cap_tokens;
    p.new_tables = new_tables;
    p.new_blocks_per_seq = new_blocks_per_seq;
    p.new_lens = new_lens;
    p.new_weights = new_weights;
    p.new_weight_stride = new_weight_stride;
    p.new_weight_cols = new_weight_cols;
    p.kept = kept;
    p.num_seqs = num_seqs;
    p.keep = keep;
    p.recent = recent;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.pool[0] = static_cast<uint4*>(k_pool);
    p.pool[1] = static_cast<uint4*>(v_pool);
    p.row_vec = (int)(row_bytes / 16);
    // K and V of a part of a row: 2 KB of each per warp and token, or the row
    p.row_lanes = 32;
    while (p.row_lanes > 1 && p.row_lanes / 2 >= p.row_vec) p.row_lanes /= 2;
    const int vec = p.row_vec > 64 ? 4 : (p.row_vec > 32 ? 2 : 1);
    p.parts = (p.row_vec + p.row_lanes * vec - 1) / (p.row_lanes * vec);
    p.errors = dev->errors;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    // More CTAs per sequence while they find idle SMs and 4096 tokens each
    // (GB300, 4 sequences of 32768 tokens: 45 us with one CTA each).
    p.select_ctas = 1;
    while (p.select_ctas < pkv::kEvictCluster &&
           2LL * p.select_ctas * num_seqs <= dev->sm_count &&
           p.cap_tokens >= 8192LL * p.select_ctas)
        p.select_ctas *= 2;
    static unsigned long long select_mask = 0;
    const long long own = ((long long)p.cap_tokens + p.select_ctas - 1) / p.select_ctas + 1024;
    p.staged = own < pkv::kEvictStaged ? (int)own : pkv::kEvictStaged;
    const size_t smem = (size_t)p.staged * sizeof(uint32_t);
    e = pkv::ensure_smem_limit(reinterpret_cast<const void*>(&pkv::evict_select_kernel),
                               &select_mask, smem);
    if (e != cudaSuccess) return cuda_fail(e);
    {
        cudaLaunchConfig_t cfg;
        std::memset(&cfg, 0, sizeof(cfg));
        cudaLaunchAttribute attr[1];
        cfg.gridDim = dim3((unsigned)(num_seqs * p.select_ctas));
        cfg.blockDim = dim3(pkv::kEvictThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = cs;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)p.select_ctas;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = p.select_ctas > 1 ? 1 : 0;
        if ((e = cudaLaunchKernelEx(&cfg, pkv::evict_select_kernel, p)) != cudaSuccess)
            return cuda_fail(e);
    }
    // Units of 32 tokens, shorter ones until the warps that are resident (3
    // CTAs per SM) get sixteen each: SMs copy at different rates, and CTAs of
    // short units start where one has ended (64 sequences cut to 1024 tokens of
    // 8 KB rows, 310 us at two units a warp, 286 at sixteen).  Below four tokens
    // a unit's table lookups weigh more than that (4 sequences cut to 8192
    // tokens of 2 KB rows, 60.6 us at four, 62.2 at one), unless there are not
    // two units for each warp (64 tokens of 1 KB rows on 16 warps took 23 us, on
    // 256 5 us).
    const int warps = pkv::kEvictCopyThreads / 32;
    const long long resident = 3LL * dev->sm_count * warps, cap = 64LL * dev->sm_count;
    p.batch = 32;
    auto count = [&] { return (long long)num_seqs * ((keep + p.batch - 1) / p.batch) * p.parts; };
    while (p.batch > 1 && count() < (p.batch > 4 ? 16 : 2) * resident) p.batch /= 2;
    long long ctas = (count() + warps - 1) / warps;
    if (ctas > cap) ctas = cap;
    const dim3 grid((unsigned)ctas);
    const int threads = pkv::kEvictCopyThreads;
    e = vec == 4   ? launch_dependent(pkv::evict_copy_kernel<4>, grid, threads, 0, cs, p)
        : vec == 2 ? launch_dependent(pkv::evict_copy_kernel<2>, grid, threads, 0, cs, p)
                   : launch_dependent(pkv::evict_copy_kernel<1>, grid, threads, 0, cs, p);
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

}  // extern "C"
