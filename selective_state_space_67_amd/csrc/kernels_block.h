// Host-side interface between the front end of the norms around a block
// (api_block.cpp) and their kernels (gated_norm.hip, block_norm.hip). Not
// installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch_limits.h"
#include "log.h"

namespace ssm {

constexpr int kMaxRow = 16384;  // elements of a row that a workgroup can hold

// Rows that share weights (and the sums of their gradients): `groups` of `rows` each, a
// group cut into `parts`, a workgroup each.
struct RowGroups {
  int64_t rows;
  int groups, parts;
};

struct GatedPlan {
  int64_t tokens;
  int H, d, in_bf16, out_bf16, gate_first, w_per_head;
  const void* x;
  const void* z;
  int64_t xs, zs;  // elements between tokens
  const float* w;
  void* out;
  const void* dout;
  void* dx;
  void* dz;
  float* dw;
  float eps;
};
hipError_t launch_gated_norm(const GatedPlan& plan, hipStream_t stream);
// Workgroups of the backward: rows of d sums in its workspace.
int64_t gated_norm_bwd_blocks(int64_t tokens, int H, int d, bool w_per_head);
hipError_t launch_gated_norm_bwd(const GatedPlan& plan, float* workspace, hipStream_t stream);

struct BlockPlan {
  int64_t B, L;
  int D, in_bf16, out_bf16, res_bf16, post, gate_rows;
  const void* y;
  int64_t ys;
  const void* x;  // null: the stream starts here
  const float* w;
  const float* w_post;
  const float* gate;  // (D), or (B, D) with gate_rows
  void* out;
  void* x_out;
  const void* dout;
  const void* dx_out;
  void* dy;
  void* dx;
  float* dw;
  float* dw_post;
  float* dgate;
  float eps, scale;
};
hipError_t launch_block_norm(const BlockPlan& plan, hipStream_t stream);
// Workgroups of the backward: rows of 3 D sums in its workspace.
int64_t block_norm_bwd_blocks(int64_t B, int64_t L, int D, bool gate_rows);
hipError_t launch_block_norm_bwd(const BlockPlan& plan, float* workspace, hipStream_t stream);

// Sums over the rows of a backward's workspace, `width` floats each, in a fixed order
// (row_sums.hip): to[g, e] = sum over the rows of group g of part[row, offset + e].
struct RowSum {
  float* to;  // null: nothing
  int64_t offset, rows_group;
  int groups;
};
hipError_t launch_row_sums(const float* part, int64_t width, int size, const RowSum (&sums)[3], hipStream_t stream);

}  // namespace ssm
