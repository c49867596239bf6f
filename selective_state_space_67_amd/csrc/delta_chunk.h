// Arguments and device code shared by the chunked passes of the gated delta
// rule: delta_chunk.hip (forward) and delta_chunk_bwd.hip (backward).
#pragma once

#include "delta_mfma.h"
#include "kernels_delta.h"

namespace ssm {

// Per (batch row, value head) and chunk the preparation leaves a record in the
// workspace: T = (I + A)^-1, P = M o QK^T and the chunk's scalars; for the backward
// T, T^T, P^T and the scalars.
constexpr int kRecT = 0, kRecP = kTriBytes, kRecGates = 2 * kTriBytes;
constexpr int kRecBytes = kRecGates + kGateFloats * 4;
constexpr int kRecTt = kTriBytes, kRecPt = 2 * kTriBytes, kRecGatesBwd = 3 * kTriBytes;
constexpr int kRecBytesBwd = kRecGatesBwd + kGateFloatsBwd * 4;

struct ChunkArgs {
  int64_t L;
  int Hk, Hv, dk, dv, group;
  int chunks;
  const void* q;
  const void* k;
  const void* v;
  int64_t qs, ks, vs;
  const void* dt;
  const void* br;
  const float* dt_bias;
  const float* A;
  const uint8_t* reset;
  float scale, beta_scale;
  bool vec;       // rows of q and k come as whole 16-byte runs of 8 entries
  char* records;  // (bh, chunk)
};

// The chunk's scalars by one wave, a lane per token, into `out` (LDS). The sums are taken
// in double and kept in two floats, so that differences of them keep a small decay's
// precision next to large ones.
template <typename InT>
__device__ __forceinline__ void chunk_gates(const ChunkArgs& a, int b, int h, int chunk, float* out, int lane) {
  const int64_t t = static_cast<int64_t>(chunk) * kChunk + lane;
  const bool valid = t < a.L;
  double g = 0.0;
  float beta = 0.0f, delta = 0.0f, slope = 0.0f;
  bool start = false;
  if (valid) {
    const int64_t i = (static_cast<int64_t>(b) * a.L + t) * a.Hv + h;
    const float raw = load_elem(static_cast<const InT*>(a.dt), i) + (a.dt_bias ? a.dt_bias[h] : 0.0f);
    delta = softplus_f32(raw);
    slope = fast_rcp(1.0f + fast_exp2(-raw * kLog2e));
    beta = a.beta_scale * fast_rcp(1.0f + fast_exp2(-load_elem(static_cast<const InT*>(a.br), i) * kLog2e));
    start = a.reset && a.reset[static_cast<int64_t>(b) * a.L + t];
    // a step's decay below 2^-16384 is 0 in float32 whatever its exponent; a NaN stays one
    if (!start) {
      g = static_cast<double>(a.A[h]) * delta * 1.4426950408889634;
      if (g < -16384.0) g = -16384.0;
    }
  }
  const uint64_t starts = __ballot(start);
  const int seg = __popcll(starts & (~uint64_t{0} >> (63 - lane)));
  bool cut = start;
#pragma unroll
  for (int off = 1; off < 64; off *= 2) {
    const double before = __shfl_up(g, off);
    const bool cut_before = __shfl_up(static_cast<int>(cut), off);
    if (lane >= off) {
      if (!cut) g += before;
      cut = cut || cut_before;
    }
  }
  const double last = __shfl(g, 63);
  const float hi = static_cast<float>(g);
  out[kE0 + lane] = seg == 0 ? fast_exp2(hi) : 0.0f;
  out[kEC + lane] = seg == __popcll(starts) ? fast_exp2(static_cast<float>(last - g)) : 0.0f;
  out[kBeta + lane] = beta;
  out[kSlope + lane] = slope;
  out[kSumHi + lane] = hi;
  out[kSumLo + lane] = static_cast<float>(g - hi);
  out[kSeg + lane] = static_cast<float>(seg);
  out[kDelta + lane] = delta;
}

// A lane's share of the sums for elements of 16 x 16 tiles in the D layout: of the four
// tokens that its rows are, or of the one that its column is.
struct RowDecay {
  f32x4 hi, lo, beta, seg;
};
struct ColDecay {
  float hi, lo, beta, seg;
};
__device__ __forceinline__ RowDecay row_decay(const float* s, int first) {
  return RowDecay{*reinterpret_cast<const f32x4*>(s + kSumHi + first), *reinterpret_cast<const f32x4*>(s + kSumLo + first),
                  *reinterpret_cast<const f32x4*>(s + kBeta + first), *reinterpret_cast<const f32x4*>(s + kSeg + first)};
}
__device__ __forceinline__ ColDecay col_decay(const float* s, int token) {
  return ColDecay{s[kSumHi + token], s[kSumLo + token], s[kBeta + token], s[kSeg + token]};
}
// exp(G_row - G_col), for a row at or after the column, or the reverse; 0 across documents.
__device__ __forceinline__ float decay_down(const RowDecay& a, int r, const ColDecay& b) {
  const float e = fast_exp2((a.hi[r] - b.hi) + (a.lo[r] - b.lo));
  return a.seg[r] == b.seg ? e : 0.0f;
}
__device__ __forceinline__ float decay_up(const RowDecay& a, int r, const ColDecay& b) {
  const float e = fast_exp2((b.hi - a.hi[r]) + (b.lo - a.lo[r]));
  return a.seg[r] == b.seg ? e : 0.0f;
}

inline bool delta_aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// Token rows of q and k come as whole 16-byte runs of 8 entries (two of them for float32).
inline bool delta_vec(const DeltaPlan& p) {
  const int64_t per = p.in_bf16 ? 8 : 4;
  return p.dk % 8 == 0 && p.qs % per == 0 && p.ks % per == 0 && delta_aligned(p.q, 16) && delta_aligned(p.k, 16);
}

inline ChunkArgs chunk_args(const DeltaPlan& p, int chunks) {
  ChunkArgs a{};
  a.L = p.L;
  a.Hk = p.Hk;
  a.Hv = p.Hv;
  a.dk = p.dk;
  a.dv = p.dv;
  a.group = p.Hv / p.Hk;
  a.chunks = chunks;
  a.q = p.q;
  a.k = p.k;
  a.v = p.v;
  a.qs = p.qs;
  a.ks = p.ks;
  a.vs = p.vs;
  a.dt = p.dt;
  a.br = p.br;
  a.dt_bias = p.dt_bias;
  a.A = p.A;
  a.reset = p.reset;
  a.scale = p.scale;
  a.beta_scale = p.beta_scale;
  a.vec = delta_vec(p);
  return a;
}

// Row tiles of 32 that hold dk: 1, 2, 3, 4, 6 or 8.
inline int padded_ks(int dk) {
  const int ks = (dk + 31) / 32;
  return ks <= 4 ? ks : ks <= 6 ? 6 : 8;
}

constexpr int kMaxLds = 160 * 1024;

// Prepare every chunk (delta_chunk.hip); bwd: the backward's records.
hipError_t launch_chunk_prepare(const DeltaPlan& p, const ChunkArgs& a, bool bwd, hipStream_t stream);

// dH at the ends of the pieces (in the starts' place), from the aggregates whose N the
// reverse walk left.
hipError_t launch_delta_fold_back(const DeltaPlan& p, const DeltaChunks& plan, char* ws, const float* dh_last,
                                  hipStream_t stream);
// The forward walk over prepared backward records that keeps every chunk's first
// state (bh, chunk, 32 padded_ks(dk), cols) and U (bh, chunk, 64, cols), cols = dv
// rounded up to 16; columns at or past dv and rows of padding are finite.
hipError_t launch_delta_states(const DeltaPlan& p, const ChunkArgs& c, const DeltaChunks& plan, char* ws, float* states,
                               float* U, hipStream_t stream);

}  // namespace ssm
