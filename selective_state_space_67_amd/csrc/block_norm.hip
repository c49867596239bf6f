// What happens between two blocks: the output y of one joins the residual
// stream x, and the input of the next is normed; and the gradients.
//
//   m = w_post y r(y), or y;  k = scale gate;  x' = x + k m;  out = w x' r(x')
//   r(v) = (mean v^2 + eps)^-1/2
//
//   dX = r (w dout - n mean(w dout n)) + dx_out with n = x' r(x'),  dw = sum dout n
//   dx = dX,  dm = k dX,  dgate = scale sum m dX,  dw_post = sum dm y r(y)
//   dy = dm, or back through the post norm
//
// One pass over the data each way: a token's row is read once, kept in registers
// and written once, so memory bounds both: 8192 rows of 2560, bfloat16 with a float32
// stream, 45.8 us for 252 MB, 5.5 TB/s (x' partly stays in the last-level cache; a large
// copy reaches 5.2), backward 74.5 us for 377 MB, 5.1, and 4.8 for the sums. Rows above
// 8192 entries outgrow the backward's registers: 206 to 286 us for as many elements, odd ones
// 377 to 699; of odd ones above 4096 it takes 120 to 196, with a bfloat16 stream 166 to 277. out is the norm of x' before x' is
// rounded to the residual stream's type, and the backward works x' out again from
// x and y, so that neither sees that rounding.
#include <utility>

#include "norm_rows.h"

namespace ssm {
namespace {

struct BlockArgs {
  RowGroups g;
  int D, out_bf16, res_bf16, post, gate_rows;
  const void* y;
  int64_t ys;
  const void* x;
  const float* w;
  const float* w_post;
  const float* gate;
  void* out;
  void* x_out;
  const void* dout;
  const void* dx_out;
  void* dy;
  void* dx;
  float* part;
  float eps, scale, share;
};

template <typename InT, typename ResT, int V, int TR, int NV, int MOST>
__global__ __launch_bounds__(MOST) void block_norm_fwd(const BlockArgs a) {
  __shared__ float lds[2][16];
  TeamSum<TR> sum;
  const Columns<V, TR, NV> c(a.D);
  const int group = RowWalk::group(a.g);
  const RowWalk walk = RowWalk::of<TR>(a.g);
  Raw<V, InT> raw_y[NV];
  Raw<V, ResT> rx[NV];
  auto load = [&](int64_t i) {
    const int64_t row = group * a.g.rows + i;
    c.load(a.y, row * a.ys, raw_y);
    if (a.x) c.load(a.x, row * a.D, rx);
  };
  using Hold = Holds<V, NV, MOST, false>;
  if (Hold::kAhead && walk.row < walk.end) load(walk.row);
  float w[NV][V], wp[NV][V], k[NV][V];
  c.weights(a.w, w);
  if (a.post) c.weights(a.w_post, wp);
  c.weights(a.gate ? a.gate + static_cast<int64_t>(group) * a.D : nullptr, k);
  for (int64_t i = walk.row; i < walk.end; i += walk.step) {
    const int64_t row = group * a.g.rows + i;
    if (!Hold::kAhead) load(i);
    float y[NV][V], x[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        y[j][e] = raw_y[j].at(e);
        x[j][e] = a.x ? rx[j].at(e) : 0.0f;
      }
    if (Hold::kAhead && i + walk.step < walk.end) load(i + walk.step);
    if (a.post) {
      const float ry = __builtin_amdgcn_rsqf(__builtin_fmaf(sum(dot(y, y), lds), a.share, a.eps));
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) y[j][e] *= ry * wp[j][e];
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float f = a.scale * k[j][e];
        y[j][e] = __builtin_fmaf(f, y[j][e], x[j][e]);
      }
    if (a.x_out) c.store(a.x_out, row * a.D, a.res_bf16, y);
    const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(sum(dot(y, y), lds), a.share, a.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) y[j][e] *= r * w[j][e];
    c.store(a.out, row * a.D, a.out_bf16, y);
  }
}

template <typename InT, typename ResT, int V, int TR, int NV, int MOST>
__global__ __launch_bounds__(MOST) void block_norm_bwd(const BlockArgs a) {
  extern __shared__ float sums[];
  __shared__ float lds[2][16];
  TeamSum<TR> sum;
  const Columns<V, TR, NV> c(a.D);
  const int group = RowWalk::group(a.g);
  const RowWalk walk = RowWalk::of<TR>(a.g);
  Raw<V, InT> raw_y[NV], rdn[NV];
  Raw<V, ResT> rx[NV], rdx[NV];
  auto load = [&](int64_t i) {
    const int64_t row = group * a.g.rows + i;
    c.load(a.y, row * a.ys, raw_y);
    if (a.x) c.load(a.x, row * a.D, rx);
    c.load(a.dout, row * a.D, rdn);
    if (a.dx_out) c.load(a.dx_out, row * a.D, rdx);
  };
  using Hold = Holds<V, NV, MOST, true>;
  if (Hold::kAhead && walk.row < walk.end) load(walk.row);
  const float* gate = a.gate ? a.gate + static_cast<int64_t>(group) * a.D : nullptr;
  float w[NV][V], wp[NV][V], k[NV][V], dw[NV][V] = {}, dwp[NV][V] = {}, dg[NV][V] = {};
  if (Hold::kWeights) {
    c.weights(a.w, w);
    if (a.post) c.weights(a.w_post, wp);
    c.weights(gate, k);
  }
  // a row of one entry has nothing across its own direction: 1 - n^2 = eps r^2 there
  const bool alone = V == 1 && a.D == 1;
  for (int64_t i = walk.row; i < walk.end; i += walk.step) {
    const int64_t row = group * a.g.rows + i;
    if (!Hold::kAhead) load(i);
    float y[NV][V], x[NV][V], dn[NV][V], dX[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        y[j][e] = raw_y[j].at(e);
        x[j][e] = a.x ? rx[j].at(e) : 0.0f;
        dn[j][e] = rdn[j].at(e);
        dX[j][e] = a.dx_out ? rdx[j].at(e) : 0.0f;
      }
    if (Hold::kAhead && i + walk.step < walk.end) load(i + walk.step);
    float ry = 1.0f;
    if (a.post) {
      ry = __builtin_amdgcn_rsqf(__builtin_fmaf(sum(dot(y, y), lds), a.share, a.eps));
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) y[j][e] *= ry;  // normed from here on
    }
    if (!Hold::kWeights) {
      if (a.post) c.weights(a.w_post, wp);
      c.weights(gate, k);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float f = a.scale * k[j][e], m = a.post ? y[j][e] * wp[j][e] : y[j][e];
        x[j][e] = __builtin_fmaf(f, m, x[j][e]);
      }
    const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(sum(dot(x, x), lds), a.share, a.eps));
    if (!Hold::kWeights) c.weights(a.w, w);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[j][e] *= r;
        dw[j][e] = __builtin_fmaf(dn[j][e], x[j][e], dw[j][e]);
        dn[j][e] *= w[j][e];
      }
    const float along = sum(dot(dn, x), lds) * a.share;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float back = alone ? r * dn[j][e] * (a.eps * r * r) : r * __builtin_fmaf(-x[j][e], along, dn[j][e]);
        dX[j][e] += back;
      }
    if (a.dx) c.store(a.dx, row * a.D, a.res_bf16, dX);
    if (!Hold::kWeights) {
      if (a.post) c.weights(a.w_post, wp);
      c.weights(gate, k);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float m = a.post ? y[j][e] * wp[j][e] : y[j][e];
        if (a.gate) dg[j][e] = __builtin_fmaf(a.scale * m, dX[j][e], dg[j][e]);
        dX[j][e] *= a.scale * k[j][e];  // dm
      }
    if (a.post) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          dwp[j][e] = __builtin_fmaf(dX[j][e], y[j][e], dwp[j][e]);
          dX[j][e] *= wp[j][e];
        }
      const float across = sum(dot(dX, y), lds) * a.share;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e)
          dX[j][e] = alone ? ry * dX[j][e] * (a.eps * ry * ry) : ry * __builtin_fmaf(-y[j][e], across, dX[j][e]);
    }
    c.store(a.dy, row * a.D, a.out_bf16, dX);
  }
  if (!a.part) return;
  float* to = a.part + static_cast<int64_t>(blockIdx.x) * 3 * a.D;
  store_sums(c, dw, sums, to);
  if (a.post) store_sums(c, dwp, sums, to + a.D);
  if (a.gate) store_sums(c, dg, sums, to + 2 * a.D);
}

BlockArgs block_args(const BlockPlan& p) {
  BlockArgs a{};
  a.g.groups = p.gate_rows ? static_cast<int>(p.B) : 1;
  a.g.rows = p.gate_rows ? p.L : p.B * p.L;
  a.D = p.D;
  a.out_bf16 = p.out_bf16;
  a.res_bf16 = p.res_bf16;
  a.post = p.post;
  a.gate_rows = p.gate_rows;
  a.y = p.y;
  a.ys = p.ys;
  a.x = p.x;
  a.w = p.w;
  a.w_post = p.w_post;
  a.gate = p.gate;
  a.out = p.out;
  a.x_out = p.x_out;
  a.dout = p.dout;
  a.dx_out = p.dx_out;
  a.dy = p.dy;
  a.dx = p.dx;
  a.eps = p.eps;
  a.scale = p.scale;
  a.share = 1.0f / static_cast<float>(p.D);
  return a;
}

template <typename InT, typename ResT>
struct Forward {
  static constexpr bool kMany = false;
  template <int V, int TR, int NV, int MOST>
  static hipError_t run(int threads, BlockArgs a, hipStream_t stream) {
    a.g.parts = row_parts(a.g, threads, TR ? threads / (TR ? TR : 1) : 1);
    const unsigned blocks = static_cast<unsigned>(a.g.groups) * a.g.parts;
    SSM_LOG("launch block_norm_fwd<%d entries a run, %d lanes a row, %d runs a lane>: grid %u x %d threads", V,
            TR ? TR : threads, NV, blocks, threads);
    hipLaunchKernelGGL((block_norm_fwd<InT, ResT, V, TR, NV, MOST>), dim3(blocks), dim3(threads), 0, stream, a);
    return hipGetLastError();
  }
};

template <typename InT, typename ResT>
struct Backward {
  static constexpr bool kMany = true;
  template <int V, int TR, int NV, int MOST>
  static hipError_t run(int threads, BlockArgs a, int parts, hipStream_t stream) {
    a.g.parts = parts;
    const unsigned blocks = static_cast<unsigned>(a.g.groups) * parts;
    const size_t lds = TR ? static_cast<size_t>(threads / (TR ? TR : 1)) * a.D * sizeof(float) : 0;
    SSM_LOG("launch block_norm_bwd<%d entries a run, %d lanes a row, %d runs a lane>: grid %u x %d threads", V,
            TR ? TR : threads, NV, blocks, threads);
    hipLaunchKernelGGL((block_norm_bwd<InT, ResT, V, TR, NV, MOST>), dim3(blocks), dim3(threads), lds, stream, a);
    return hipGetLastError();
  }
};

template <template <typename, typename> class F, typename... X>
hipError_t pick_types(const BlockPlan& p, X&&... x) {
  bool runs = p.D % 8 == 0 && p.ys % 8 == 0;
  for (const void* q : {p.y, p.x, static_cast<const void*>(p.w), static_cast<const void*>(p.w_post),
                        static_cast<const void*>(p.gate), static_cast<const void*>(p.out),
                        static_cast<const void*>(p.x_out), p.dout, p.dx_out, static_cast<const void*>(p.dy),
                        static_cast<const void*>(p.dx)})
    runs = runs && aligned_to(q, 16);
  if (p.in_bf16)
    return p.res_bf16 ? pick_team<F<bf16_t, bf16_t>>(runs, p.D, p.B * p.L, std::forward<X>(x)...)
                      : pick_team<F<bf16_t, float>>(runs, p.D, p.B * p.L, std::forward<X>(x)...);
  return p.res_bf16 ? pick_team<F<float, bf16_t>>(runs, p.D, p.B * p.L, std::forward<X>(x)...)
                    : pick_team<F<float, float>>(runs, p.D, p.B * p.L, std::forward<X>(x)...);
}

}  // namespace

hipError_t launch_block_norm(const BlockPlan& p, hipStream_t stream) {
  return pick_types<Forward>(p, block_args(p), stream);
}

int64_t block_norm_bwd_blocks(int64_t B, int64_t L, int D, bool gate_rows) {
  // 8192 rows of 2560 79 us, with 768 threads 85, with 1024 87
  return row_sum_blocks(gate_rows ? B : 1, gate_rows ? L : B * L, D, 512);
}

hipError_t launch_block_norm_bwd(const BlockPlan& p, float* workspace, hipStream_t stream) {
  BlockArgs a = block_args(p);
  const int64_t blocks = block_norm_bwd_blocks(p.B, p.L, p.D, p.gate_rows), D = p.D;
  const RowSum sums[3] = {{p.dw, 0, blocks, 1},
                          {p.post ? p.dw_post : nullptr, D, blocks, 1},
                          {p.gate ? p.dgate : nullptr, 2 * D, blocks / a.g.groups, a.g.groups}};
  a.part = sums[0].to || sums[1].to || sums[2].to ? workspace : nullptr;
  const hipError_t e = pick_types<Backward>(p, a, static_cast<int>(blocks / a.g.groups), stream);
  return e != hipSuccess ? e : launch_row_sums(workspace, 3 * D, p.D, sums, stream);
}

}  // namespace ssm
