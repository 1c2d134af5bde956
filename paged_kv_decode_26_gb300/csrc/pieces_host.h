// pieces_host.h -- host side shared by the calls built on the piece decode
// (cache_ops_capi.cu, shared_capi.cu): argument checks, workspace layout,
// launch parameters.
#pragma once

#include <cstring>

#include "capi_host.h"
#include "decode_pieces_kernel.cuh"

namespace pkv {
namespace host {

constexpr int kDefaultSms = 152;      // workspace sizes asked for without a device

struct PiecesWorkspace {
    size_t o, ml, seg_first, seg_last, end;   // byte offsets; end: first free byte
};

size_t align256(size_t n);

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// kv heads per stream: the largest of 8, 4, 2, 1 that divides n_kv_heads.
int pieces_stream_heads(int n_kv_heads);

// CTAs of the piece decode: one per SM, fewer where the longest contexts
// allowed could not give every stream its least run; and, with short_runs, CTAs
// of short runs, none where the longest contexts allowed are too short for them.
struct PiecesGrid {
    int ctas, extra;
};
PiecesGrid pieces_grid(int num_seqs, int n_kv_heads, int max_context_len, int sm_count,
                       bool short_runs);

PiecesWorkspace pieces_workspace(int num_seqs, int n_heads, int n_kv_heads, int head_dim,
                                 const PiecesGrid& grid);

// Argument checks that the calls share with paged_attn_decode.
pkv_status check_paged_decode(const void* out, pkv_dtype out_dtype, const void* q,
                              const void* k_pool, const void* v_pool, pkv_dtype kv_dtype,
                              const int32_t* block_tables, int max_blocks_per_seq,
                              const int32_t* context_lens, int num_seqs, int n_heads,
                              int n_kv_heads, int head_dim, int block_size, int num_blocks,
                              float scale, int max_context_len);

pkv_status check_workspace(const void* workspace, size_t bytes, size_t need);

// Fills p and the chunk maps.
pkv_status fill_pieces(PieceParams* p, CUtensorMap* tm_k, CUtensorMap* tm_v,
                       const PiecesGrid& grid, void* out,
                       pkv_dtype out_dtype, const void* q, const void* k_pool, const void* v_pool,
                       pkv_dtype kv_dtype, const int32_t* block_tables, int max_blocks_per_seq,
                       const int32_t* context_lens, int num_seqs, int n_heads, int n_kv_heads,
                       int head_dim, int block_size, int num_blocks, float scale,
                       int max_context_len, const PiecesWorkspace& w, void* workspace,
                       const DeviceInfo& dev);

// A kernel that starts while the one ahead of it on the stream drains (it
// waits for that one's results before it reads them).
template <class Kernel, class Params>
cudaError_t launch_dependent(Kernel kernel, dim3 grid, int threads, size_t smem,
                             cudaStream_t stream, const Params& p) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace host
}  // namespace pkv
