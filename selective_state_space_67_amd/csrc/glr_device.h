// Device code shared by the gated linear recurrence's kernels (glr_fwd.hip,
// glr_pieces.hip, glr_bwd.hip): the arguments, a step's gates, decay and
// multiplier, and rows of inputs as loaded.
//
//   s = sigmoid(dt_raw + dt_bias) or softplus(dt_raw + dt_bias)
//   a = exp(A s) (0 at a reset),  c = sqrt(1 - a^2), 1 - a or 1
//   h = a h + c i u,  i = sigmoid(in_raw + in_bias) or 1,  out = h silu(z) or h
//
// A lane owns one channel, a wave 64 neighbouring ones (128 bytes of a bfloat16
// row), and a wave's rows are its own: which row a wave is at, whether it is a
// document's first and whether it exists are the same for all of its lanes. So
// rows may start at any address and lie at any stride, and a reset costs
// branches that are taken together.
#pragma once

#include "device_math.h"
#include "kernels_glr.h"

namespace ssm {

constexpr int kLanes = 64;

struct GlrArgs {
  int64_t L;
  int D, tiles;        // tiles: groups of 64 channels
  int pieces;          // of the sequence, piece_rows each
  int64_t piece_rows;
  const void* u;
  const void* dt;
  const void* in;  // null: no input gate
  const void* z;   // null: no output gate
  int64_t us, ds, is, zs;
  const float* A;
  const float* dt_bias;
  const float* in_bias;
  const uint8_t* reset;
  const float* h0;
  void* out;
  float* h_last;
  int out_bf16;        // type of out, or of the gradients
  float* P;            // (B, pieces, D): what a piece does to the state that enters it
  float* H;
  float* G;            // and to the adjoint that enters it from behind
  float* starts;       // (B, pieces, D): state entering a piece
  float* ends;         // adjoint entering a piece from behind
  const void* dout;
  const float* dh_last;
  void* du;
  void* d_dt;
  void* d_in;
  void* dz;
  float* dh0;
  float* part;         // (B pieces, 3, D): a piece's sums for dA, d_dt_bias and din_bias
};

// An element as loaded; widened only when it is used.
__device__ __forceinline__ uint32_t raw_load(const char* row, uint32_t at, const bf16_t*) {
  return *reinterpret_cast<const uint16_t*>(row + at);
}
__device__ __forceinline__ uint32_t raw_load(const char* row, uint32_t at, const float*) {
  return *reinterpret_cast<const uint32_t*>(row + at);
}
template <typename T>
__device__ __forceinline__ float widen(uint32_t raw) {
  return __uint_as_float(sizeof(T) == 2 ? raw << 16 : raw);
}

// K rows from `row` on, of which `rows` (at least 1) exist; the last one stands in for the others.
template <typename T, int K>
__device__ __forceinline__ void load_rows(const void* base, int64_t row, int64_t stride, int rows, uint32_t at,
                                          uint32_t (&x)[K]) {
  const char* p = static_cast<const char*>(base) + row * stride * static_cast<int64_t>(sizeof(T));
  const int64_t step = stride * static_cast<int64_t>(sizeof(T));
#pragma unroll
  for (int k = 0; k < K; ++k) {
    x[k] = raw_load(p, at, static_cast<const T*>(nullptr));
    p += k + 1 < rows ? step : 0;
  }
}

// Which of K rows are a document's first: one bit each, the same in all lanes.
template <int K>
__device__ __forceinline__ uint32_t reset_byte(const uint8_t* reset, int64_t row, int rows, int lane) {
  return reset && lane < K && lane < rows ? reset[row + lane] : 0;
}

__device__ __forceinline__ float sigmoid_f32(float x) { return fast_rcp(1.0f + fast_exp2(-x * kLog2e)); }

template <int DECAY>
__device__ __forceinline__ float decay_gate(float raw) {
  return DECAY == kGlrSigmoid ? sigmoid_f32(raw) : softplus_f32(raw);
}

// a = e^g and c. Near g = 0, where long memories live, 1 - a comes from the series of
// expm1 (to x^6; the next term is below 5e-8 of it) and a from 1 - (1 - a), so that both
// keep float32's precision: e^g itself has an error of 1e-7 there, which over a thousand
// steps adds up, and 1 - e^g loses what the memory's length is made of.
template <int MIX>
__device__ __forceinline__ void decay_terms(float g, float& a, float& c) {
  const float E = fast_exp2(g * kLog2e);
  float p = __builtin_fmaf(g, 1.0f / 720.0f, 1.0f / 120.0f);
  p = __builtin_fmaf(g, p, 1.0f / 24.0f);
  p = __builtin_fmaf(g, p, 1.0f / 6.0f);
  p = __builtin_fmaf(g, p, 0.5f);
  p = __builtin_fmaf(g, p, 1.0f);
  const float lost = -g * p;
  const bool near = fabsf(g) < 0.25f;
  a = near ? 1.0f - lost : E;
  if constexpr (MIX == kGlrOne) {
    c = 1.0f;
  } else {
    const float e = near ? lost : 1.0f - E;
    c = MIX == kGlrRest ? e : __builtin_amdgcn_sqrtf(__builtin_fmaf(e, a, e));  // 1 - a^2 = (1 - a) (1 + a)
  }
}

// What a run of steps does to a state is h -> P h + H. A run with a document's start in it
// has the sign bit of P set (P is never negative otherwise): the state from before it is
// not looked at then, since 0 times an infinite one would be NaN.
constexpr float kCut = -0.0f;
__device__ __forceinline__ float through(float P, float H, float h) {
  return __float_as_int(P) < 0 ? H : __builtin_fmaf(P, h, H);
}

// Results: rounding to bfloat16 is to nearest even, by the hardware's conversion (a NaN stays one).
__device__ __forceinline__ uint16_t to_bf16(float x) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}
__device__ __forceinline__ void store_result(char* row, uint32_t channel, float x, bool bf16) {
  if (bf16)
    *reinterpret_cast<uint16_t*>(row + 2 * channel) = to_bf16(x);
  else
    *reinterpret_cast<float*>(row + 4 * channel) = x;
}

}  // namespace ssm
