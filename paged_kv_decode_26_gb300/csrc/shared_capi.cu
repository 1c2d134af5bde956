// shared_capi.cu -- paged_attn_decode_shared of the C ABI: validation, the
// cut of the work into prefix items and runs, workspace layout and launches
// (decode_shared_kernel.cuh, then the merge).  Declarations and contracts:
// pagedkv.h.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>

#include "attn_host.h"
#include "capi_host.h"
#include "decode_shared_launch.h"
#include "pieces_host.h"

using namespace pkv::host;

namespace {

// A split costs its key tiles and about this many more (queries, first and
// last products, output of the partial states).
constexpr int kSplitCost = 4;

// Whether the prefixes are attended once per group: where they fill a key tile
// and the other members' reads of them, at most, come to 24 MB.  Below that every
// member reads its whole context, which saves a launch.  GB300, GPU time of a
// call (and with the launches from Python), each member alone against once per
// group: 0.4 MB 11.3 (22) / 12.5 us (25); 16 MB 13.3 (22) / 14.9 (26); 31 MB 17.9
// (22) / 14.2 (24), eight groups 18.7 / 20.6; 66 MB 21.3 / 17.8, of prefixes of 64
// tokens 25.3 / 27.2; 251 MB 39.4 / 22.2, of 64 tokens 77.1 / 73.3.
constexpr double kSharedLeast = 24e6;
bool prefix_once(int num_seqs, int num_groups, int max_group, int max_prefix, int n_kv_heads,
                 int head_dim) {
    const long long members = std::min((long long)num_seqs, (long long)num_groups * max_group);
    const long long again = max_group > 0 ? members - (members + max_group - 1) / max_group : 0;
    const double bytes = 4.0 * n_kv_heads * head_dim * max_prefix * again;
    const bool pays = max_prefix >= pkv::kAtKeys && bytes >= kSharedLeast;
    return tuning(PKV_TUNE_SHARED_PREFIX, pays ? 1 : 0) != 0;
}

struct SharedShape {
    int split_tokens;
    int max_splits;
    PiecesGrid grid;      // of the rest of the contexts
    PiecesWorkspace pieces;
    size_t start, pre_o, pre_ml, end;
};

SharedShape shared_shape(int num_seqs, int num_groups, int max_group, int max_prefix, int n_heads,
                         int n_kv_heads, int head_dim, int max_context_len, int sm_count) {
    SharedShape c;
    const int G = n_heads / n_kv_heads;
    const int pair_rows = 2 * pkv::kAtRows / G;
    const int pairs = max_group > 0 ? (max_group + pair_rows - 1) / pair_rows : 0;
    const long long units = (long long)num_groups * n_kv_heads * pairs;
    c.max_splits = 0;
    c.split_tokens = pkv::kAtKeys;
    if (units > 0 && max_prefix > 0 &&
        prefix_once(num_seqs, num_groups, max_group, max_prefix, n_kv_heads, head_dim)) {
        // Work items (split x kv head x pair of row tiles x group) are dealt
        // out to the SMs in turn: the split length with the smallest sum of
        // key tiles over the busiest SM's items, the longer one of equals.
        // Of the lengths that give s splits the shortest, ceil(tiles / s), is
        // the best; a cost of s splits is at least units (tiles + kSplitCost s)
        // / SMs, so more splits are tried only while that is below the best
        // (a few hundred at most, whatever the bound of the prefixes).
        const long long tiles = ((long long)max_prefix + pkv::kAtKeys - 1) / pkv::kAtKeys;
        long long best = 0;
        for (long long s = 1; s <= tiles && (best == 0 || units * (tiles + kSplitCost * s) <
                                                              best * sm_count);) {
            const long long n = (tiles + s - 1) / s;
            const long long cost = (units * s + sm_count - 1) / sm_count * (n + kSplitCost);
            if (best == 0 || cost < best) {
                best = cost;
                c.split_tokens = (int)(n * pkv::kAtKeys);
            }
            // the next number of splits that some length gives
            s = n > 1 ? (tiles + n - 2) / (n - 1) : tiles + 1;
        }
        c.max_splits = (int)(((long long)max_prefix + c.split_tokens - 1) / c.split_tokens);
    }
    // (no short runs to take over: the prefixes fill the SMs that end early)
    c.grid = pieces_grid(num_seqs, n_kv_heads, max_context_len, sm_count, false);
    c.pieces = pieces_workspace(num_seqs, n_heads, n_kv_heads, head_dim, c.grid);
    const size_t rows = (size_t)num_seqs * n_heads * c.max_splits;
    c.start = c.pieces.end;
    c.pre_o = align256(c.start + (size_t)num_seqs * sizeof(int));
    c.pre_ml = align256(c.pre_o + rows * head_dim * sizeof(float));
    c.end = align256(c.pre_ml + rows * 2 * sizeof(float));
    return c;
}

bool groups_ok(int num_seqs, int num_groups, int max_group, int max_prefix, int max_context_len) {
    return num_groups >= 0 && max_group >= 0 && max_group <= num_seqs && max_prefix >= 0 &&
           max_prefix <= max_context_len;
}

}  // namespace

extern "C" {

PKV_API size_t pkv_decode_shared_workspace_bytes(int num_seqs, int num_groups, int max_group,
                                                 int max_prefix, int n_heads, int n_kv_heads,
                                                 int head_dim, int block_size,
                                                 int max_context_len) {
    if (!supported_shape(n_heads, n_kv_heads, head_dim, block_size) || num_seqs <= 0 ||
        max_context_len < 0 ||
        !groups_ok(num_seqs, num_groups, max_group, max_prefix, max_context_len))
        return 0;
    DeviceInfo* dev = nullptr;
    const int sms = device_info(&dev) == cudaSuccess ? dev->sm_count : kDefaultSms;
    return shared_shape(num_seqs, num_groups, max_group, max_prefix, n_heads, n_kv_heads, head_dim,
                        max_context_len, sms)
        .end;
}

PKV_API pkv_status paged_attn_decode_shared(
    void* out, pkv_dtype out_dtype, const void* q, const void* k_pool, const void* v_pool,
    pkv_dtype kv_dtype, const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, const int32_t* group_start, const int32_t* prefix_lens,
    int num_groups, int max_group, int max_prefix, int num_seqs, int n_heads, int n_kv_heads,
    int head_dim, int block_size, int num_blocks, float scale, int max_context_len,
    void* workspace, size_t workspace_bytes, void* stream) {
    pkv_status st = check_paged_decode(out, out_dtype, q, k_pool, v_pool, kv_dtype, block_tables,
                                       max_blocks_per_seq, context_lens, num_seqs, n_heads,
                                       n_kv_heads, head_dim, block_size, num_blocks, scale,
                                       max_context_len);
    if (st != PKV_OK) return st;
    if (num_groups < 0 || max_group < 0 || max_prefix < 0) return invalid("group sizes");
    if (num_groups > 65535) return unsupported("more than 65535 groups");
    if (num_seqs == 0) return PKV_OK;
    if (num_groups > 0 && (!group_start || !prefix_lens))
        return invalid("group_start or prefix_lens is NULL");
    if (!aligned4(group_start) || !aligned4(prefix_lens))
        return invalid("group_start and prefix_lens must be 4-byte aligned");
    if (!groups_ok(num_seqs, num_groups, max_group, max_prefix, max_context_len))
        return invalid("max_group beyond num_seqs, or max_prefix beyond max_context_len");
    DeviceInfo* dev = nullptr;
    cudaError_t e = device_info(&dev);
    if (e != cudaSuccess) return cuda_fail(e);
    const SharedShape c = shared_shape(num_seqs, num_groups, max_group, max_prefix, n_heads,
                                       n_kv_heads, head_dim, max_context_len, dev->sm_count);
    if ((st = check_workspace(workspace, workspace_bytes, c.end)) != PKV_OK) return st;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    pkv::SharedLaunch L;
    std::memset(&L, 0, sizeof(L));
    L.stream = static_cast<cudaStream_t>(stream);
    pkv::PieceParams& p = L.p;
    st = fill_pieces(&p, &L.tm_kc, &L.tm_vc, c.grid, out, out_dtype, q, k_pool, v_pool, kv_dtype,
                     block_tables, max_blocks_per_seq, context_lens, num_seqs, n_heads,
                     n_kv_heads, head_dim, block_size, num_blocks, scale, max_context_len,
                     c.pieces, workspace, *dev);
    if (st != PKV_OK) return st;
    p.group_start = group_start;
    p.prefix_lens = prefix_lens;
    p.num_groups = num_groups;
    p.max_group = max_group;
    p.max_prefix = max_prefix;
    p.start = reinterpret_cast<int*>(ws + c.start);
    p.pre_o = reinterpret_cast<float*>(ws + c.pre_o);
    p.pre_ml = reinterpret_cast<float*>(ws + c.pre_ml);
    p.split_tokens = c.split_tokens;
    const bool once = c.max_splits > 0 && num_blocks > 0;
    p.max_splits = once ? c.max_splits : 0;

    // ---- the prefixes (not once: whole contexts, nothing to join)
    const int G = n_heads / n_kv_heads;
    pkv::AttnParams& a = L.a;
    if (once) {
        const long long unit = (long long)head_dim * sizeof(float) * c.max_splits;
        if ((e = encode_rows_map(&L.tm_q, q, kv_dtype, num_seqs, n_heads, head_dim,
                                 (long long)n_heads * head_dim, G, pkv::kAtRows / G)) ||
            (e = encode_pool_map(&L.tm_k, k_pool, kv_dtype, num_blocks, block_size, n_kv_heads,
                                 head_dim, 1, true)) ||
            (e = encode_pool_map(&L.tm_v, v_pool, kv_dtype, num_blocks, block_size, n_kv_heads,
                                 head_dim, 1, true)) ||
            (e = encode_out_map(&L.tm_o, ws + c.pre_o, PKV_F32, num_seqs, n_heads, unit / 128, unit,
                                unit * n_heads, G)))
            return cuda_fail(e);
        a.out_dtype = out_dtype;
        a.num_seqs = num_seqs;
        a.n_heads = n_heads;
        a.n_kv_heads = n_kv_heads;
        a.group = G;
        a.scale_log2 = p.scale_log2;
        a.stages = attn_stages(head_dim, dev->smem_optin);
        a.row_tiles = pkv::attn_row_tiles(out_dtype == PKV_F32);
        const int item_rows = a.row_tiles * pkv::kAtRows / G;
        a.tiles = (max_group + item_rows - 1) / item_rows;
        a.group_start = group_start;
        a.prefix_lens = prefix_lens;
        a.max_group = max_group;
        a.max_prefix = max_prefix;
        a.block_tables = block_tables;
        a.max_blocks_per_seq = max_blocks_per_seq;
        a.context_lens = context_lens;
        a.cap_tokens = p.cap_tokens;
        a.block_size = block_size;
        a.num_blocks = num_blocks;
        a.split_tokens = c.split_tokens;
        a.max_splits = c.max_splits;
        a.pre_o = reinterpret_cast<float*>(ws + c.pre_o);
        a.pre_ml = reinterpret_cast<float*>(ws + c.pre_ml);
        a.errors = dev->errors;
        a.n_items = (long long)num_groups * n_kv_heads * a.tiles * c.max_splits;
        // (as for prompts; beyond that many candidates most may be empty)
        a.dynamic = a.n_items > dev->sm_count && a.n_items <= 16 * dev->sm_count;
        L.prefix_ctas = (int)(a.dynamic || a.n_items < dev->sm_count ? a.n_items : dev->sm_count);
    }
    const bool precise = out_dtype == PKV_F32;
    e = kv_dtype == PKV_BF16 ? pkv::launch_shared_bf16(head_dim, precise, L)
                             : pkv::launch_shared_f16(head_dim, precise, L);
    if (e != cudaSuccess) return cuda_fail(e);
    // Pieces of a row to expect: the prefix's splits, and the cuts of the rest.
    // Up to 12 one warp merges them (GB300, 8192 rows of 6 pieces: 13 us, 17 us
    // with four warps a row).
    const long long streams = (long long)c.grid.ctas * (pkv::kPieceWarps / p.stream_heads);
    const long long pairs = (long long)num_seqs * (n_kv_heads / p.stream_heads);
    const bool few = p.max_splits + 2 + streams / pairs <= 12;
    const int rows = few ? pkv::kFinishWarps : 1;
    const dim3 grid((unsigned)((n_heads + rows - 1) / rows), (unsigned)num_seqs);
    auto merge = head_dim == 128 ? (few ? pkv::decode_shared_finish_kernel<128, 1>
                                        : pkv::decode_shared_finish_kernel<128, 4>)
                                 : (few ? pkv::decode_shared_finish_kernel<64, 1>
                                        : pkv::decode_shared_finish_kernel<64, 4>);
    e = launch_dependent(merge, grid, pkv::kFinishThreads, 0, L.stream, p);
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
}

}  // extern "C"
