// The norm of a mixer's output with its gate, and its gradients:
//
//   r(v) = (mean v^2 + eps)^-1/2,  y = w x r(x) silu(z),  or  y = w v r(v) with v = x silu(z)
//
//   back through a norm: dn -> r (dn - n mean(dn n)),  n = v r(v)
//
// One pass over the data each way: a row (a head of a token) is read once, kept in
// registers and written once, so memory bounds both: 8 x 2048 tokens of 12 heads of 128
// 27.3 us for 151 MB, 5.5 TB/s (the output partly stays in the last-level cache; a large
// copy reaches 5.2); backward of 8192 rows of 5120 82.8 us for 419 MB, 5.1, and 5.0 for
// the sums. A team per head and not a wave: 64 lanes of 16 bytes each hold four heads of
// 128 (with a wave for each, 80 us).
#include <utility>

#include "norm_rows.h"

namespace ssm {
namespace {

struct GatedArgs {
  RowGroups g;
  int H, d, out_bf16, gate_first, w_per_head;
  const void* x;
  const void* z;
  int64_t xs, zs;
  const float* w;
  void* out;
  const void* dout;
  void* dx;
  void* dz;
  float* part;
  float eps, share;
};

// Row i of a group: (token, head), and where it lies in dense tensors.
struct GatedRow {
  int64_t x, z, dense;
  __device__ __forceinline__ GatedRow(const GatedArgs& a, int64_t i, int group) {
    const int64_t token = a.w_per_head ? i : i / a.H;
    const int64_t head = a.w_per_head ? group : i - token * a.H;
    x = token * a.xs + head * a.d;
    z = token * a.zs + head * a.d;
    dense = (token * a.H + head) * a.d;
  }
};

template <typename InT, int V, int TR, int NV, int MOST>
__global__ __launch_bounds__(MOST) void gated_norm_fwd(const GatedArgs a) {
  __shared__ float lds[2][16];
  TeamSum<TR> sum;
  const Columns<V, TR, NV> c(a.d);
  const int group = RowWalk::group(a.g);
  const RowWalk walk = RowWalk::of<TR>(a.g);
  Raw<V, InT> rx[NV], rz[NV];
  auto load = [&](int64_t i) {
    const GatedRow row(a, i, group);
    c.load(a.x, row.x, rx);
    c.load(a.z, row.z, rz);
  };
  using Hold = Holds<V, NV, MOST, false>;
  if (Hold::kAhead && walk.row < walk.end) load(walk.row);
  float w[NV][V];
  c.weights(a.w ? a.w + (a.w_per_head ? static_cast<int64_t>(group) * a.d : 0) : nullptr, w);
  for (int64_t i = walk.row; i < walk.end; i += walk.step) {
    if (!Hold::kAhead) load(i);
    float x[NV][V], z[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[j][e] = rx[j].at(e);
        z[j][e] = silu_f32(rz[j].at(e));
        if (a.gate_first) {
          x[j][e] *= z[j][e];
          z[j][e] = 1.0f;
        }
      }
    if (Hold::kAhead && i + walk.step < walk.end) load(i + walk.step);
    const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(sum(dot(x, x), lds), a.share, a.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) x[j][e] = x[j][e] * r * w[j][e] * z[j][e];
    c.store(a.out, GatedRow(a, i, group).dense, a.out_bf16, x);
  }
}

template <typename InT, int V, int TR, int NV, int MOST>
__global__ __launch_bounds__(MOST) void gated_norm_bwd(const GatedArgs a) {
  extern __shared__ float sums[];
  __shared__ float lds[2][16];
  TeamSum<TR> sum;
  const Columns<V, TR, NV> c(a.d);
  const int group = RowWalk::group(a.g);
  const RowWalk walk = RowWalk::of<TR>(a.g);
  Raw<V, InT> rx[NV], rz[NV], rdy[NV];
  auto load = [&](int64_t i) {
    const GatedRow row(a, i, group);
    c.load(a.x, row.x, rx);
    c.load(a.z, row.z, rz);
    c.load(a.dout, row.dense, rdy);
  };
  using Hold = Holds<V, NV, MOST, false>;
  if (Hold::kAhead && walk.row < walk.end) load(walk.row);
  const float* weight = a.w ? a.w + (a.w_per_head ? static_cast<int64_t>(group) * a.d : 0) : nullptr;
  float w[NV][V], dw[NV][V] = {};
  if (Hold::kWeights) c.weights(weight, w);
  for (int64_t i = walk.row; i < walk.end; i += walk.step) {
    if (!Hold::kAhead) load(i);
    float x[NV][V], z[NV][V], dy[NV][V], n[NV][V];
    float slope[NV][V];  // of silu at z, whose value replaces z
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[j][e] = rx[j].at(e);
        z[j][e] = rz[j].at(e);
        dy[j][e] = rdy[j].at(e);
        const float s = fast_rcp(1.0f + fast_exp2(-z[j][e] * kLog2e));
        slope[j][e] = s * __builtin_fmaf(z[j][e], 1.0f - s, 1.0f);
        z[j][e] *= s;
        n[j][e] = a.gate_first ? x[j][e] * z[j][e] : x[j][e];
      }
    if (Hold::kAhead && i + walk.step < walk.end) load(i + walk.step);
    const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(sum(dot(n, n), lds), a.share, a.eps));
    if (!Hold::kWeights) c.weights(weight, w);
    // dy becomes the gradient of the normed row, and with the norm first the gate's is taken on the way
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        n[j][e] *= r;
        const float wn = w[j][e] * n[j][e];
        if (a.gate_first) {
          dw[j][e] = __builtin_fmaf(dy[j][e], n[j][e], dw[j][e]);
          dy[j][e] *= w[j][e];
        } else {
          const float through = dy[j][e] * z[j][e];
          dw[j][e] = __builtin_fmaf(through, n[j][e], dw[j][e]);
          slope[j][e] *= dy[j][e] * wn;  // dz
          dy[j][e] = through * w[j][e];
        }
      }
    const float along = sum(dot(dy, n), lds) * a.share;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        // a row of one entry has nothing across its own direction: 1 - n^2 = eps r^2 there
        const float dv = V == 1 && a.d == 1 ? r * dy[j][e] * (a.eps * r * r)
                                            : r * __builtin_fmaf(-n[j][e], along, dy[j][e]);
        if (a.gate_first) {
          slope[j][e] *= dv * x[j][e];  // dz
          dy[j][e] = dv * z[j][e];
        } else {
          dy[j][e] = dv;
        }
      }
    const int64_t at = GatedRow(a, i, group).dense;
    c.store(a.dx, at, a.out_bf16, dy);
    c.store(a.dz, at, a.out_bf16, slope);
  }
  if (a.part) store_sums(c, dw, sums, a.part + static_cast<int64_t>(blockIdx.x) * a.d);
}

GatedArgs gated_args(const GatedPlan& p) {
  GatedArgs a{};
  a.g.groups = p.w_per_head ? p.H : 1;
  a.g.rows = p.w_per_head ? p.tokens : p.tokens * p.H;
  a.H = p.H;
  a.d = p.d;
  a.out_bf16 = p.out_bf16;
  a.gate_first = p.gate_first;
  a.w_per_head = p.w_per_head;
  a.x = p.x;
  a.z = p.z;
  a.xs = p.xs;
  a.zs = p.zs;
  a.w = p.w;
  a.out = p.out;
  a.dout = p.dout;
  a.dx = p.dx;
  a.dz = p.dz;
  a.eps = p.eps;
  a.share = 1.0f / static_cast<float>(p.d);
  return a;
}

template <typename InT>
struct Forward {
  static constexpr bool kMany = false;
  template <int V, int TR, int NV, int MOST>
  static hipError_t run(int threads, GatedArgs a, hipStream_t stream) {
    a.g.parts = row_parts(a.g, threads, TR ? threads / (TR ? TR : 1) : 1);
    const unsigned blocks = static_cast<unsigned>(a.g.groups) * a.g.parts;
    SSM_LOG("launch gated_norm_fwd<%d entries a run, %d lanes a row, %d runs a lane>: grid %u x %d threads", V,
            TR ? TR : threads, NV, blocks, threads);
    hipLaunchKernelGGL((gated_norm_fwd<InT, V, TR, NV, MOST>), dim3(blocks), dim3(threads), 0, stream, a);
    return hipGetLastError();
  }
};

template <typename InT>
struct Backward {
  static constexpr bool kMany = false;
  template <int V, int TR, int NV, int MOST>
  static hipError_t run(int threads, GatedArgs a, int parts, hipStream_t stream) {
    a.g.parts = parts;
    const unsigned blocks = static_cast<unsigned>(a.g.groups) * parts;
    const size_t lds = TR ? static_cast<size_t>(threads / (TR ? TR : 1)) * a.d * sizeof(float) : 0;
    SSM_LOG("launch gated_norm_bwd<%d entries a run, %d lanes a row, %d runs a lane>: grid %u x %d threads", V,
            TR ? TR : threads, NV, blocks, threads);
    hipLaunchKernelGGL((gated_norm_bwd<InT, V, TR, NV, MOST>), dim3(blocks), dim3(threads), lds, stream, a);
    return hipGetLastError();
  }
};

bool in_runs(const GatedPlan& p) {
  return p.d % 8 == 0 && p.xs % 8 == 0 && p.zs % 8 == 0 && aligned_to(p.x, 16) && aligned_to(p.z, 16) &&
         aligned_to(p.w, 16) && aligned_to(p.out, 16) && aligned_to(p.dout, 16) && aligned_to(p.dx, 16) &&
         aligned_to(p.dz, 16);
}

}  // namespace

hipError_t launch_gated_norm(const GatedPlan& p, hipStream_t stream) {
  const GatedArgs a = gated_args(p);
  const int64_t rows = p.tokens * p.H;
  if (p.in_bf16) return pick_team<Forward<bf16_t>>(in_runs(p), p.d, rows, a, stream);
  return pick_team<Forward<float>>(in_runs(p), p.d, rows, a, stream);
}

int64_t gated_norm_bwd_blocks(int64_t tokens, int H, int d, bool w_per_head) {
  // 8 x 2048 x 10 heads of 128 and 2048 of 2048: 44 us and 46, with 512 threads 49 and 54, with 1024 50 and 45
  return row_sum_blocks(w_per_head ? H : 1, w_per_head ? tokens : tokens * H, d, 768);
}

hipError_t launch_gated_norm_bwd(const GatedPlan& p, float* workspace, hipStream_t stream) {
  GatedArgs a = gated_args(p);
  a.part = p.dw ? workspace : nullptr;
  const int parts = static_cast<int>(gated_norm_bwd_blocks(p.tokens, p.H, p.d, p.w_per_head) / a.g.groups);
  const int64_t rows = p.tokens * p.H;
  const hipError_t e = p.in_bf16 ? pick_team<Backward<bf16_t>>(in_runs(p), p.d, rows, a, parts, stream)
                                 : pick_team<Backward<float>>(in_runs(p), p.d, rows, a, parts, stream);
  if (e != hipSuccess) return e;
  return launch_row_sums(workspace, p.d, p.d, {{p.dw, 0, parts, a.g.groups}, {}, {}}, stream);
}

}  // namespace ssm
