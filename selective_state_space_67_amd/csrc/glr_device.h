// Device code shared by the gated linear recurrence's kernels (glr_fwd.hip,
// glr_chain.hip, glr_pieces.hip, glr_bwd.hip): the arguments, a step's gates, decay and
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
  int pieces;          // of the sequence (backward)
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

// A tensor's rows from a wave's first one on, through a buffer descriptor: the lanes' offsets
// stay in one register and a row's is a scalar, so that an access takes no vector arithmetic
// (with 64-bit addresses a third of the walk's vector instructions went into them).
struct RowBuffer {
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t step;  // bytes from row to row; K of them stay below 2^31 (kGlrMaxStride)
  __device__ __forceinline__ RowBuffer(const void* base, int64_t row, int64_t stride, int size)
      : rsrc(__builtin_amdgcn_make_buffer_rsrc(
            const_cast<char*>(static_cast<const char*>(base) + row * stride * size), 0, 0x7fffffff, 0x00020000)),
        step(static_cast<uint32_t>(stride) * size) {}
};

// An element as loaded; widened only when it is used.
template <typename T>
__device__ __forceinline__ uint32_t raw_load(const RowBuffer& b, uint32_t at, uint32_t row) {
  if constexpr (sizeof(T) == 2)
    return __builtin_amdgcn_raw_buffer_load_b16(b.rsrc, at, row * b.step, 0);
  else
    return __builtin_amdgcn_raw_buffer_load_b32(b.rsrc, at, row * b.step, 0);
}
template <typename T>
__device__ __forceinline__ float widen(uint32_t raw) {
  return __uint_as_float(sizeof(T) == 2 ? raw << 16 : raw);
}

// K rows from `row` on, of which `rows` (at least 1) exist; the last one stands in for the others.
template <typename T, int K>
__device__ __forceinline__ void load_rows(const void* base, int64_t row, int64_t stride, int rows, uint32_t at,
                                          uint32_t (&x)[K]) {
  const RowBuffer b(base, row, stride, sizeof(T));
#pragma unroll
  for (int k = 0; k < K; ++k) x[k] = raw_load<T>(b, at, min(k, rows - 1));
}

// What K rows of a wave do to a state that enters them (P, H) and to an adjoint that enters
// from behind (P, G), as below. `rows` exist; `cuts` start a document. With PLAIN all exist and
// none does.
template <bool PLAIN, bool BWD, int K>
__device__ __forceinline__ void run_rows(const float (&a)[K], const float (&b)[K], const float (&dy)[K], int rows,
                                         uint32_t cuts, float& P, float& H, float& G, bool& cut) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (PLAIN || k < rows) {
      const bool here = !PLAIN && ((cuts >> k) & 1);
      cut |= here;
      P *= a[k];
      H = here ? b[k] : __builtin_fmaf(a[k], H, b[k]);
      // what lies behind a document's start is out of the adjoint's sight
      if (BWD && !cut) G = __builtin_fmaf(P, dy[k], G);
    }
  }
}

// K rows of results, of which `rows` exist (all with PLAIN): rounding to bfloat16 is to nearest even, by the
// hardware's conversion (a NaN stays one).
template <bool PLAIN, int K>
__device__ __forceinline__ void store_rows(void* base, int64_t row, int D, int rows, uint32_t channel, bool bf16,
                                           const float (&x)[K]) {
  const RowBuffer b(base, row, D, bf16 ? 2 : 4);
  const uint32_t at = (bf16 ? 2 : 4) * channel;
  auto store = [&](int k) {
    if (bf16)
      __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, static_cast<__bf16>(x[k])), b.rsrc, at,
                                            k * b.step, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[k]), b.rsrc, at, k * b.step, 0);
  };
  if (PLAIN || rows == K) {
#pragma unroll
    for (int k = 0; k < K; ++k) store(k);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < rows) store(k);
  }
}

// Which of K rows are a document's first, a lane each.
template <int K>
__device__ __forceinline__ uint32_t reset_byte(const uint8_t* reset, int64_t row, int rows, int lane) {
  return reset && lane < K && lane < rows ? reset[row + lane] : 0;
}

__device__ __forceinline__ float sigmoid_f32(float x) { return fast_rcp(1.0f + fast_exp2(-x * kLog2e)); }

// A channel's constants. The sigmoids' biases come ready for the exponential of base 2.
template <int DECAY>
struct Channel {
  float A, dt, in;
  bool far;  // some of the wave's channels may have |A s| >= 1/4 (sigmoid: s is at most 1)
  __device__ __forceinline__ Channel(const GlrArgs& g, int ch)
      : A(g.A[ch]), dt(g.dt_bias ? g.dt_bias[ch] : 0.0f), in(g.in_bias ? -kLog2e * g.in_bias[ch] : 0.0f) {
    if (DECAY == kGlrSigmoid) dt *= -kLog2e;
    far = __builtin_amdgcn_ballot_w64(!(fabsf(A) < 0.25f)) != 0;
  }
};

// A value loaded before a loop that prefetches: waited for here. Taken as under way, its first
// use in the loop would wait in every round for whatever was loaded last.
__device__ __forceinline__ void arrived(float& x) { asm volatile("" : "+v"(x)); }

// sigmoid(x + bias), with `bias` times -log2 e
__device__ __forceinline__ float biased_sigmoid(float x, float bias) {
  return fast_rcp(1.0f + fast_exp2(__builtin_fmaf(x, -kLog2e, bias)));
}

// sigmoid(x) from -x log2 e, and e^-x. 1 - sigmoid(x) is their product, which keeps its digits where
// the sigmoid is near 1: taken from the rounded sigmoid it would be off by up to 2^-25, all of it from
// x = 17 on. (An infinite e^-x belongs to a sigmoid of 0.)
struct Sigmoid {
  float e, value;
  __device__ __forceinline__ explicit Sigmoid(float x) : e(fast_exp2(x)), value(fast_rcp(1.0f + e)) {}
};

// The gate s, and (sigmoid) the e that makes e s = 1 - s.
template <int DECAY>
__device__ __forceinline__ float decay_gate(float raw, const Channel<DECAY>& c, float& e) {
  if (DECAY == kGlrSoftplus) return softplus_f32(raw + c.dt);
  const Sigmoid s(__builtin_fmaf(raw, -kLog2e, c.dt));
  e = s.e;
  return s.value;
}

// a = e^g and c. Near g = 0, where long memories live, 1 - a comes from the series of
// expm1 (to x^6; the next term is below 5e-8 of it) and a from 1 - (1 - a), so that both
// keep float32's precision: e^g itself has an error of 1e-7 there, which over a thousand
// steps adds up, and 1 - e^g loses what the memory's length is made of. FAR: g may be
// below -1/4.
template <int MIX, bool FAR>
__device__ __forceinline__ void decay_terms(float g, float& a, float& c) {
  float p = __builtin_fmaf(g, 1.0f / 720.0f, 1.0f / 120.0f);
  p = __builtin_fmaf(g, p, 1.0f / 24.0f);
  p = __builtin_fmaf(g, p, 1.0f / 6.0f);
  p = __builtin_fmaf(g, p, 0.5f);
  p = __builtin_fmaf(g, p, 1.0f);
  float lost = -g * p;
  a = 1.0f - lost;
  if (FAR) {
    const float E = fast_exp2(g * kLog2e);
    const bool near = fabsf(g) < 0.25f;
    a = near ? a : E;
    lost = near ? lost : 1.0f - E;
  }
  // 1 - a^2 = (1 - a) (1 + a)
  c = MIX == kGlrOne ? 1.0f : MIX == kGlrRest ? lost : __builtin_amdgcn_sqrtf(__builtin_fmaf(lost, a, lost));
}

// Gate, decay and multiplier of K rows. Whether the exponential is needed at all is the same
// for the wave: from its channels' A, or (softplus) from these rows' largest |g|.
template <typename T, int DECAY, int MIX, int K>
__device__ __forceinline__ void decays(const Channel<DECAY>& ch, const uint32_t (&dt)[K], float (&s)[K], float (&e)[K],
                                       float (&a)[K], float (&c)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = decay_gate<DECAY>(widen<T>(dt[k]), ch, e[k]);
  bool far = ch.far;
  if (DECAY == kGlrSoftplus) {
    float most = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) most = fmaxf(most, fabsf(ch.A * s[k]));
    far = __builtin_amdgcn_ballot_w64(most >= 0.25f) != 0;
  }
  if (far) {
#pragma unroll
    for (int k = 0; k < K; ++k) decay_terms<MIX, true>(ch.A * s[k], a[k], c[k]);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) decay_terms<MIX, false>(ch.A * s[k], a[k], c[k]);
  }
}

// Decays a and inputs b = c i u of K rows; cuts: those that start a document, whose c is 1.
template <typename T, int DECAY, int MIX, bool IN, int K>
__device__ __forceinline__ void terms(const Channel<DECAY>& ch, const uint32_t (&u)[K], const uint32_t (&dt)[K],
                                      const uint32_t (&in)[K], uint32_t cuts, float (&a)[K], float (&b)[K]) {
  float s[K], e[K], c[K];
  decays<T, DECAY, MIX, K>(ch, dt, s, e, a, c);
#pragma unroll
  for (int k = 0; k < K; ++k) b[k] = IN ? widen<T>(u[k]) * biased_sigmoid(widen<T>(in[k]), ch.in) : widen<T>(u[k]);
  if (MIX == kGlrOne) return;
  if (cuts) {
    keep_branch();
#pragma unroll
    for (int k = 0; k < K; ++k) c[k] = (cuts >> k) & 1 ? 1.0f : c[k];
  }
#pragma unroll
  for (int k = 0; k < K; ++k) b[k] *= c[k];
}

// What a run of steps does to a state is h -> P h + H. A run with a document's start in it
// has the sign bit of P set (P is never negative otherwise): the state from before it is
// not looked at then, since 0 times an infinite one would be NaN.
constexpr float kCut = -0.0f;
__device__ __forceinline__ float through(float P, float H, float h) {
  return __float_as_int(P) < 0 ? H : __builtin_fmaf(P, h, H);
}
// P of two runs together.
__device__ __forceinline__ float joined(float a, float b) {
  return __float_as_int(a) < 0 || __float_as_int(b) < 0 ? kCut : a * b;
}

}  // namespace ssm
