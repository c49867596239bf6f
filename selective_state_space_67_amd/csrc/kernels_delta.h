// Host-side interface between the front end of the gated delta rule and the
// head norms (api_delta.cpp) and their kernels (delta_step.hip,
// delta_chunk.hip, delta_chunk_bwd.hip, qk_norm.hip). Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch_limits.h"
#include "log.h"

namespace ssm {

// One gated delta rule launch after validation. Pointers are device pointers;
// optional ones are nullptr. Token strides are in elements.
struct DeltaPlan {
  int64_t B, L;
  int Hk, Hv, dk, dv;
  int in_bf16, out_bf16;
  const void* q;
  const void* k;
  const void* v;
  int64_t qs, ks, vs;
  const void* dt;
  const void* br;
  const float* dt_bias;
  const float* A;
  const uint8_t* reset;
  const float* h0;  // state before the first step, or null
  void* out;
  float* h_last;    // state after the last step, or null; may equal h0 in the decode window
  float scale, beta_scale;
};

// The recurrence step by step with the state in registers (delta_step.hip).
hipError_t launch_delta_steps(const DeltaPlan& plan, hipStream_t stream);

// The recurrence in chunks of 64 tokens on the matrix cores (delta_chunk.hip): how
// many chunks, the pieces the sequence is split into, and the workspace layout.
struct DeltaChunks {
  int chunks, pieces, chunks_piece;
  int groups, group_pieces;  // of pieces, where their states are folded
  size_t off_records, off_agg, off_starts, off_group_agg, off_group_starts, bytes;
  size_t off_turned;  // M^T of the pieces, which the backward keeps
};
// requested = 0: automatic. Pure host arithmetic.
DeltaChunks plan_delta_chunks(int64_t B, int64_t L, int Hv, int dk, int dv, int requested);
// Whether every launch of a forward call stays below 2^32 threads (heads: B Hv), and of a
// backward call (key_heads: B Hk).
bool delta_grids_fit(int64_t heads, int dk, int dv, const DeltaChunks& plan);
hipError_t launch_delta_chunks(const DeltaPlan& plan, const DeltaChunks& chunks, void* workspace, hipStream_t stream);

// The backward pass (delta_chunk_bwd.hip). DeltaPlan gives the forward's inputs.
struct DeltaBwdPlan {
  int grad_bf16;
  const void* dout;
  const float* dh_last;
  void* dq;
  void* dk;
  void* dv;
  void* ddt;
  void* dbr;
  float* dA;
  float* dbias;
  float* dh0;
};
struct DeltaBwdLayout {  // workspace byte offsets
  int chunks;
  DeltaChunks walk;  // the pieces of the forward walk, with offsets in this workspace
  size_t off_records, off_states, off_U, off_dstates, off_dR, off_sums, off_part, bytes;
};
DeltaBwdLayout plan_delta_bwd(int64_t B, int64_t L, int Hv, int dk, int dv);
bool delta_bwd_grids_fit(int64_t heads, int64_t key_heads, int dk, int dv, const DeltaBwdLayout& layout);
hipError_t launch_delta_bwd(const DeltaPlan& plan, const DeltaBwdPlan& grads, const DeltaBwdLayout& layout,
                            void* workspace, hipStream_t stream);

// Norms and rotation (qk_norm.hip).
struct NormPlan {
  int64_t B, L, P;
  int Hq, Hk, d, rot;
  int in_bf16, out_bf16;
  const void* q;
  const void* k;
  int64_t qs, ks;
  const float* wq;
  const float* wk;
  const float* cos;
  const float* sin;
  const int32_t* positions;
  void* q_out;
  void* k_out;
  const void* dq_out;  // backward
  const void* dk_out;
  void* dq;
  void* dk;
  float* dwq;
  float* dwk;
  float* part;  // norm_bwd_blocks() rows of 2 * d sums
  float eps;
  int l2, interleaved;
};
hipError_t launch_qk_norm(const NormPlan& plan, hipStream_t stream);
// Workgroups of the backward pass: the rows of its partial sums.
int norm_bwd_blocks(int64_t tokens, int heads, int d);
hipError_t launch_qk_norm_bwd(const NormPlan& plan, hipStream_t stream);

}  // namespace ssm
