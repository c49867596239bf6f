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
constexpr int kRecBytesBwd = kRecGatesBwd + kGateFloats * 4;

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
  char* records;  // (bh, chunk)
};

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
  return a;
}

inline bool delta_aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// Token rows of q and k come as whole 16-byte runs of 8 entries (two of them for float32).
inline bool delta_vec(const DeltaPlan& p) {
  const int64_t per = p.in_bf16 ? 8 : 4;
  return p.dk % 8 == 0 && p.qs % per == 0 && p.ks % per == 0 && delta_aligned(p.q, 16) && delta_aligned(p.k, 16);
}

// Prepare every chunk (delta_chunk.hip); bwd: the backward's records.
hipError_t launch_chunk_prepare(const DeltaPlan& p, const ChunkArgs& a, bool bwd, hipStream_t stream);

}  // namespace ssm
