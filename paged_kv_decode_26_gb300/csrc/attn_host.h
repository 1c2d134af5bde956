// attn_host.h -- host side shared by the calls built on attn_tc_kernel.cuh.
#pragma once

#include "capi_host.h"

namespace pkv {
namespace host {

// Rows [rows, heads, head_dim] (row stride in elements) as a 4-D tensor for
// TMA: dims (64, head_dim / 64, heads, rows), box (64, 1, box_heads,
// box_rows), 128-byte swizzle: one load per 64-element half brings box_rows x
// box_heads rows of 128 bytes.  Rows past the tensor read as zeros.
cudaError_t encode_rows_map(CUtensorMap* map, const void* x, pkv_dtype dt, int rows, int heads,
                            int head_dim, long long row_stride, int box_heads, int box_rows);

// Output rows [rows, heads, head_dim] for TMA stores: element (i, h, d) at
// i * row_bytes + h * head_bytes + d * es, es 2 or 4 (fp32), `parts` 128-byte
// parts per (row, head) apart by 128 bytes.  Box: one part of group heads x
// 32 / group rows, 128-byte swizzle.
cudaError_t encode_out_map(CUtensorMap* map, void* out, pkv_dtype dt, int rows, int heads,
                           long long parts, long long head_bytes, long long row_bytes, int group);

// Slots of the K/V ring that fit beside the queries.
int attn_stages(int head_dim, int smem_optin);

}  // namespace host
}  // namespace pkv
