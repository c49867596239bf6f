// The gated delta rule step by step, the state of a head held in registers:
// the decode window (ssm_delta_update) and sequences too short to pay for the
// chunked passes.
//
//   H' = a H,  u = beta (v - H'^T k),  H = H' + k u^T,  out = scale H^T q
//
// Both products with the state are taken of the state before the step, so one
// pass over its entries serves the step:
//
//   u   = beta (v - a (H^T k))
//   out = scale (a (H^T q) + (k.q) u)
//
// Columns of H (entries of v) are independent. A wave owns 16 columns of one
// head: 4 lanes of 4 columns each by 16 row groups of R consecutive rows, so a
// lane holds R x 4 entries, loads and stores them as 16-byte runs, and each
// product needs one sum over the 16 row groups (lanes of equal column), done
// with lane rotations and half-wave swaps. Four waves make a workgroup, so that
// a row's neighbouring 64-byte pieces are fetched from one CU.
//
// A decode step is bound by the state's bytes, 8 dk dv per head: 64 sequences of 16 heads of
// 128 x 128 take 21.1 us, 6.4 TB/s (the state is partly in the last-level cache when the
// steps follow one another; after a read of 1 GB between them 30 us, events included, 4.5
// TB/s); a small step by the call itself (10.3 us for one sequence of 12 heads, of which the
// kernel takes 4.2). Of several steps each takes 0.9 us, the latency of its arithmetic: the sums over
// the rows, u, and the state's update. (The next token loaded while one is worked on: 16
// steps 17.4 -> 16.0 us for 1 x 16 heads, 73 -> 80 us for 64 x 16; not kept.)
#include <algorithm>

#include "device_math.h"
#include "kernels_delta.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 16;       // columns per wave
constexpr int kColsBlock = 64;  // columns per workgroup

struct StepArgs {
  int64_t L;
  int Hv, dk, dv, group;  // group: value heads per key head
  int col_blocks;             // workgroups per head
  int out_bf16;
  const void* q;
  const void* k;
  const void* v;
  int64_t qs, ks, vs;
  const void* dt;
  const void* br;
  const float* dt_bias;
  const float* A;
  const uint8_t* reset;
  const float* h0;
  void* out;
  float* h_last;
  float scale, beta_scale;
};

// Sum over the 16 lanes of a wave that share lane % 4, in all of them.
__device__ __forceinline__ float row_group_sum(float x) {
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x124, 0xF, 0xF, true));  // row_ror:4
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x128, 0xF, 0xF, true));  // row_ror:8
  const auto s16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(s16[0]) + __uint_as_float(s16[1]);
  const auto s32 = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(s32[0]) + __uint_as_float(s32[1]);
}

// `n` consecutive elements as float; VEC: the run is whole and aligned to
// min(16, its size) bytes, otherwise entries at or past `left` read as 0.
template <typename T, int n, bool VEC>
__device__ __forceinline__ void load_run(const T* p, int left, float (&x)[n]) {
  if constexpr (VEC) {
    constexpr int per = 16 / static_cast<int>(sizeof(T)) < n ? 16 / static_cast<int>(sizeof(T)) : n;
    using R = Run<T, per>;
#pragma unroll
    for (int i = 0; i < n; i += per) {
      const typename R::raw w = R::load(p + i);
#pragma unroll
      for (int j = 0; j < per; ++j) x[i + j] = R::at(w, j);
    }
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] = i < left ? load_elem(p, i) : 0.0f;
  }
}

template <typename InT, int R, bool VEC>
__global__ __launch_bounds__(kThreads) void delta_steps(const StepArgs a) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int bh = blockIdx.x / a.col_blocks, b = bh / a.Hv, h = bh - b * a.Hv;
  const int c0 = (blockIdx.x - bh * a.col_blocks) * kColsBlock + wave * kCols + (lane % 4) * 4;
  const int r0 = (lane / 4) * R;
  const int cl = a.dv - c0, rl = a.dk - r0;  // columns and rows left
  const int hk = h / a.group;
  const int64_t state = (static_cast<int64_t>(b) * a.Hv + h) * a.dk * a.dv;

  float H[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (a.h0 && r < rl && cl > 0)
      load_run<float, 4, VEC>(a.h0 + state + static_cast<int64_t>(r0 + r) * a.dv + c0, cl, H[r]);
    else
      H[r][0] = H[r][1] = H[r][2] = H[r][3] = 0.0f;
  }
  const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
  const InT* qp = static_cast<const InT*>(a.q) + static_cast<int64_t>(b) * a.L * a.qs + static_cast<int64_t>(hk) * a.dk + r0;
  const InT* kp = static_cast<const InT*>(a.k) + static_cast<int64_t>(b) * a.L * a.ks + static_cast<int64_t>(hk) * a.dk + r0;
  const InT* vp = static_cast<const InT*>(a.v) + static_cast<int64_t>(b) * a.L * a.vs + static_cast<int64_t>(h) * a.dv + c0;
  const int64_t gate0 = static_cast<int64_t>(b) * a.L * a.Hv + h;

  for (int64_t t = 0; t < a.L; ++t) {
    float k[R], q[R], v[4];
    load_run<InT, R, VEC>(kp + t * a.ks, rl, k);
    load_run<InT, R, VEC>(qp + t * a.qs, rl, q);
    if (cl > 0)
      load_run<InT, 4, VEC>(vp + t * a.vs, cl, v);
    else
      v[0] = v[1] = v[2] = v[3] = 0.0f;
    const int64_t gi = gate0 + t * a.Hv;
    const float delta = softplus_f32(load_elem(static_cast<const InT*>(a.dt), gi) + bias);
    const float beta =
        a.beta_scale * fast_rcp(1.0f + fast_exp2(-load_elem(static_cast<const InT*>(a.br), gi) * kLog2e));
    float al = fast_exp2(A * delta * kLog2e);
    if (a.reset && a.reset[static_cast<int64_t>(b) * a.L + t]) {
      al = 0.0f;  // a document's first token carries nothing over, whatever its decay (NaN, infinite)
#pragma unroll
      for (int r = 0; r < R; ++r) H[r][0] = H[r][1] = H[r][2] = H[r][3] = 0.0f;
    }
    float kh[4] = {}, qh[4] = {}, kq = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      kq = __builtin_fmaf(k[r], q[r], kq);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        kh[c] = __builtin_fmaf(k[r], H[r][c], kh[c]);
        qh[c] = __builtin_fmaf(q[r], H[r][c], qh[c]);
      }
    }
    kq = row_group_sum(kq);
    float o[4], u[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      u[c] = beta * __builtin_fmaf(-al, row_group_sum(kh[c]), v[c]);
      o[c] = a.scale * __builtin_fmaf(al, row_group_sum(qh[c]), kq * u[c]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) H[r][c] = __builtin_fmaf(al, H[r][c], k[r] * u[c]);
    if (lane < 4 && cl > 0) {
      const int64_t oi = (gate0 + t * a.Hv) * a.dv + c0;
      if constexpr (VEC) {
        if (a.out_bf16)
          store_run<4>(static_cast<bf16_t*>(a.out) + oi, o);
        else
          store_run<4>(static_cast<float*>(a.out) + oi, o);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c >= cl) break;
          if (a.out_bf16)
            store_elem(static_cast<bf16_t*>(a.out), oi + c, o[c]);
          else
            store_elem(static_cast<float*>(a.out), oi + c, o[c]);
        }
      }
    }
  }
  if (!a.h_last) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r >= rl || cl <= 0) break;
    float* p = a.h_last + state + static_cast<int64_t>(r0 + r) * a.dv + c0;
    if constexpr (VEC) {
      store_run<4>(p, H[r]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < cl) p[c] = H[r][c];
    }
  }
}

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

template <typename InT, int R>
hipError_t launch_rows(const DeltaPlan& p, const StepArgs& a, hipStream_t stream) {
  // Whole runs: rows fill the lanes' groups exactly, columns come in fours,
  // and every run starts at a multiple of its size.
  const uintptr_t e = sizeof(InT), rows = std::min<uintptr_t>(16, R * e), cols = 4 * e;
  const bool vec = a.dk == 16 * R && a.dv % 4 == 0 && aligned_to(a.h0, 16) && aligned_to(a.h_last, 16) &&
                   aligned_to(a.q, rows) && aligned_to(a.k, rows) && aligned_to(a.v, cols) &&
                   (a.qs * e) % rows == 0 && (a.ks * e) % rows == 0 && (a.vs * e) % cols == 0 &&
                   aligned_to(a.out, a.out_bf16 ? 8 : 16);
  const dim3 grid(static_cast<unsigned>(p.B * a.Hv * a.col_blocks));
  SSM_LOG("launch delta_steps<%d rows per lane, whole runs %d>: %s in; grid %u x %d threads", R, vec,
          sizeof(InT) == 2 ? "bf16" : "f32", grid.x, kThreads);
  if (vec)
    hipLaunchKernelGGL((delta_steps<InT, R, true>), grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((delta_steps<InT, R, false>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <typename InT>
hipError_t launch_dtype(const DeltaPlan& p, const StepArgs& a, hipStream_t stream) {
  if (a.dk <= 32) return launch_rows<InT, 2>(p, a, stream);
  if (a.dk <= 64) return launch_rows<InT, 4>(p, a, stream);
  if (a.dk <= 128) return launch_rows<InT, 8>(p, a, stream);
  return launch_rows<InT, 16>(p, a, stream);
}

}  // namespace

hipError_t launch_delta_steps(const DeltaPlan& p, hipStream_t stream) {
  StepArgs a{};
  a.L = p.L;
  a.Hv = p.Hv;
  a.dk = p.dk;
  a.dv = p.dv;
  a.group = p.Hv / p.Hk;
  a.col_blocks = (p.dv + kColsBlock - 1) / kColsBlock;
  a.out_bf16 = p.out_bf16;
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
  a.h0 = p.h0;
  a.out = p.out;
  a.h_last = p.h_last;
  a.scale = p.scale;
  a.beta_scale = p.beta_scale;
  return p.in_bf16 ? launch_dtype<bf16_t>(p, a, stream) : launch_dtype<float>(p, a, stream);
}

}  // namespace ssm
