// Host-side interface between the front end of the gated linear recurrence
// (api_glr.cpp) and its kernels (glr_fwd.hip, glr_chain.hip, glr_pieces.hip,
// glr_bwd.hip). Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch_limits.h"
#include "log.h"

namespace ssm {

constexpr int kGlrSigmoid = 0, kGlrSoftplus = 1;         // decay
constexpr int kGlrUnit = 0, kGlrRest = 1, kGlrOne = 2;   // mix

// Elements between tokens stay below this, so that a wave's rows can be reached by 32-bit offsets.
constexpr int64_t kGlrMaxStride = int64_t{1} << 24;

// One call after validation. Pointers are device pointers; optional ones are
// nullptr. Token strides are in elements.
struct GlrPlan {
  int64_t B, L, D;
  int in_bf16, out_bf16, decay, mix;  // out_bf16: type of out, or of the gradients
  const void* u;
  const void* dt;
  const void* in;
  const void* z;
  int64_t us, ds, is, zs;
  const float* A;
  const float* dt_bias;
  const float* in_bias;
  const uint8_t* reset;
  const float* h0;
  void* out;
  float* h_last;  // may equal h0 in the decode window
  // backward
  const void* dout;
  const float* dh_last;
  void* du;
  void* d_dt;
  void* d_in;
  void* dz;
  float* dA;
  float* d_dt_bias;
  float* din_bias;
  float* dh0;
};

// How a sequence is cut into pieces, and where the workspace holds what joins them.
struct GlrPieces {
  int64_t pieces, rows;  // rows of a piece; forward, pieces = 1: one walk from end to end, no workspace
  int waves;             // of a workgroup that takes a piece of 64 channels
  int64_t segments;      // of pieces, for the backward's fold
  int each;              // pieces of a segment
  size_t off_P, off_H, off_G, off_starts, off_ends, off_part, off_segments, bytes;
};
// Pure host arithmetic, like the others here.
GlrPieces plan_glr(int64_t B, int64_t L, int64_t D);
GlrPieces plan_glr_bwd(int64_t B, int64_t L, int64_t D);
// Whether every launch of a call stays below 2^32 threads.
bool glr_grids_fit(int64_t B, int64_t D, const GlrPieces& pieces);
// Sequences that go step by step, one thread a channel.
bool glr_by_steps(int64_t L);
bool glr_steps_fit(int64_t B, int64_t D);

hipError_t launch_glr(const GlrPlan& plan, const GlrPieces& pieces, void* workspace, hipStream_t stream);
hipError_t launch_glr_steps(const GlrPlan& plan, hipStream_t stream);
hipError_t launch_glr_bwd(const GlrPlan& plan, const GlrPieces& pieces, void* workspace, hipStream_t stream);

// Between the kernels' files: the forward in pieces that follow each other on the chip
// (glr_chain.hip), and the backward's first two passes (glr_pieces.hip).
GlrPieces plan_glr_chain(int64_t B, int64_t L, int64_t D);
hipError_t launch_glr_chain(const GlrPlan& plan, const GlrPieces& pieces, void* workspace, hipStream_t stream);
struct GlrArgs;
GlrArgs glr_args(const GlrPlan& plan);
hipError_t launch_glr_aggregates(const GlrPlan& plan, const GlrArgs& args, hipStream_t stream);
hipError_t launch_glr_fold(const GlrPlan& plan, const GlrArgs& args, const GlrPieces& pieces, float* segments,
                           hipStream_t stream);
// A piece of the backward is 8 rows for each of this many waves.
constexpr int kGlrBwdWaves = 4;
// Pieces of a segment, where the backward's fold goes in segments.
constexpr int kGlrSegment = 64;

}  // namespace ssm
