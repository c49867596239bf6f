// What joins the pieces of a sequence in the gated linear recurrence: the pairs
// of what each piece does to a state, and the states that enter the pieces.
//
// A piece maps the state h that enters it to P h + H, and (backward) the
// adjoint m that enters it from behind to P m + G, with P the product of its
// decays and
//   H = the state it leaves from zero,   G = sum_t (prod_{r <= t} a_r) dout_t silu(z_t)
// A workgroup makes a piece's three values for 64 channels, its waves those of
// equal parts of the rows; the fold runs the same scheme over the pieces that the
// walk runs over rows.
#include "glr_device.h"
#include "glr_launch.h"

namespace ssm {
namespace {

constexpr int kAggWaves = 8, kAggRows = 8;
constexpr int kFoldWaves = 16, kFoldRows = 8;

template <typename InT, int DECAY, int MIX, bool IN, bool Z, bool BWD, int W, int K>
__global__ __launch_bounds__(W * kLanes) void glr_aggregate(const GlrArgs g, const int count) {
  __shared__ float ex[3][W][kLanes];
  const int lane = threadIdx.x % kLanes, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int tile = blockIdx.x % g.tiles, rest = blockIdx.x / g.tiles;
  const int piece = rest % count, batch = rest / count;
  const int channel = tile * kLanes + lane, ch = min(channel, g.D - 1);
  const uint32_t at = static_cast<uint32_t>(ch) * sizeof(InT);
  const int64_t row0 = batch * g.L;
  // the wave's rows (a piece has a multiple of W K; the last one's waves may have none)
  const int part = static_cast<int>(g.piece_rows) / W;
  const int begin = static_cast<int>(piece * g.piece_rows) + w * part;
  const int end = min(static_cast<int>(g.L), begin + part);
  const Channel<DECAY> c(g, ch);
  float P = 1.0f, H = 0.0f, G = 0.0f;
  bool cut = false;
  uint32_t u[K], dt[K], in[K], z[K], rdy[K], reset;
  auto load = [&](int t) {
    const int rows = min(K, end - t);
    load_rows<InT, K>(g.dt, row0 + t, g.ds, rows, at, dt);
    if (IN) load_rows<InT, K>(g.in, row0 + t, g.is, rows, at, in);
    load_rows<InT, K>(g.u, row0 + t, g.us, rows, at, u);
    if (BWD) load_rows<InT, K>(g.dout, row0 + t, g.D, rows, at, rdy);
    if (BWD && Z) load_rows<InT, K>(g.z, row0 + t, g.zs, rows, at, z);
    reset = reset_byte<K>(g.reset, row0 + t, rows, lane);
  };
  if (begin < end) load(begin);
  for (int t = begin; t < end; t += K) {
    const int rows = min(K, end - t);
    const uint32_t cuts = static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(reset != 0));
    float a[K], b[K], dy[K];
    terms<InT, DECAY, MIX, IN, K>(c, u, dt, in, cuts, a, b);
    if (BWD) {
#pragma unroll
      for (int k = 0; k < K; ++k) dy[k] = Z ? widen<InT>(rdy[k]) * silu_f32(widen<InT>(z[k])) : widen<InT>(rdy[k]);
    }
    if (t + K < end) load(t + K);
    if (rows == K && cuts == 0 && !cut)
      run_rows<true, BWD, K>(a, b, dy, K, 0, P, H, G, cut);
    else
      run_rows<false, BWD, K>(a, b, dy, rows, cuts, P, H, G, cut);
  }
  ex[0][w][lane] = cut ? kCut : P;
  ex[1][w][lane] = H;
  if (BWD) ex[2][w][lane] = G;
  __syncthreads();
  if (w >= (BWD ? 3 : 2) || channel >= g.D) return;
  // wave 0 joins the P, wave 1 the H, wave 2 the G
  const int64_t to = (static_cast<int64_t>(batch) * g.pieces + piece) * g.D + ch;
  if (w == 0) {
    P = 1.0f;
    cut = false;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      cut |= __float_as_int(ex[0][i][lane]) < 0;
      P *= ex[0][i][lane];
    }
    g.P[to] = cut ? kCut : P;
  } else if (w == 1) {
    H = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) H = through(ex[0][i][lane], ex[1][i][lane], H);
    g.H[to] = H;
  } else {
    G = 0.0f;
#pragma unroll
    for (int i = W - 1; i >= 0; --i) G = through(ex[0][i][lane], ex[2][i][lane], G);
    g.G[to] = G;
  }
}

// States entering the pieces (forward: from h0 on), or adjoints entering them from
// behind (backward: from dh_last on, the last piece first). A workgroup takes 64
// channels of a batch row, its waves K pieces each.
template <bool BACK>
__device__ __forceinline__ void fold_pieces(const GlrArgs& g, int64_t count, int64_t batch, int ch, bool on, int lane,
                                            int w, float2 (*pairs)[kFoldWaves][kLanes]) {
  constexpr int W = kFoldWaves, K = kFoldRows;
  const int64_t base = batch * g.pieces * g.D + ch;
  const float* add = BACK ? g.G : g.H;
  float* to = BACK ? g.ends : g.starts;
  const float* first = BACK ? g.dh_last : g.h0;
  float h = first ? first[batch * g.D + ch] : 0.0f;
  int buf = 0;
  for (int64_t i0 = 0; i0 < count; i0 += W * K, buf ^= 1) {
    float a[K], b[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = i0 + w * K + k;
      const int64_t from = base + (BACK ? count - 1 - i : i) * g.D;
      a[k] = i < count ? g.P[from] : 1.0f;
      b[k] = i < count ? add[from] : 0.0f;
    }
    float P = 1.0f, H = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      H = through(a[k], b[k], H);
      P = __float_as_int(a[k]) < 0 || __float_as_int(P) < 0 ? kCut : P * a[k];
    }
    pairs[buf][w][lane] = make_float2(P, H);
    __syncthreads();
    float mine = h;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 p = pairs[buf][i][lane];
      mine = i == w ? h : mine;
      h = through(p.x, p.y, h);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = i0 + w * K + k;
      if (on && i < count) to[base + (BACK ? count - 1 - i : i) * g.D] = mine;
      mine = through(a[k], b[k], mine);
    }
  }
  if (w != 0 || !on) return;
  if (BACK) {
    if (g.dh0) g.dh0[batch * g.D + ch] = h;
  } else if (count < g.pieces) {
    to[base + count * g.D] = h;
  }
}

__global__ __launch_bounds__(kFoldWaves * kLanes) void glr_fold(const GlrArgs g, const int64_t count, const int ways) {
  __shared__ float2 pairs[2][kFoldWaves][kLanes];
  const int lane = threadIdx.x % kLanes, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int way = blockIdx.x % ways, rest = blockIdx.x / ways;
  const int tile = rest % g.tiles;
  const int64_t batch = rest / g.tiles;
  const int channel = tile * kLanes + lane, ch = min(channel, g.D - 1);
  const bool on = channel < g.D;
  if (way == 0)
    fold_pieces<false>(g, count, batch, ch, on, lane, w, pairs);
  else
    fold_pieces<true>(g, count, batch, ch, on, lane, w, pairs);
}

struct Aggregate {
  template <typename InT, int DECAY, int MIX, bool IN, bool Z>
  static hipError_t run(unsigned blocks, const GlrArgs& g, int count, bool backward, hipStream_t stream) {
    if (backward)
      hipLaunchKernelGGL((glr_aggregate<InT, DECAY, MIX, IN, Z, true, kGlrBwdWaves, kAggRows>), dim3(blocks),
                         dim3(kGlrBwdWaves * kLanes), 0, stream, g, count);
    else
      hipLaunchKernelGGL((glr_aggregate<InT, DECAY, MIX, IN, false, false, kAggWaves, kAggRows>), dim3(blocks),
                         dim3(kAggWaves * kLanes), 0, stream, g, count);
    return hipGetLastError();
  }
};

}  // namespace

GlrArgs glr_args(const GlrPlan& p, const GlrPieces& q, void* workspace) {
  GlrArgs g{};
  g.L = p.L;
  g.D = static_cast<int>(p.D);
  g.tiles = (g.D + kLanes - 1) / kLanes;
  g.pieces = static_cast<int>(q.pieces);
  g.piece_rows = q.rows;
  g.u = p.u;
  g.dt = p.dt;
  g.in = p.in;
  g.z = p.z;
  g.us = p.us;
  g.ds = p.ds;
  g.is = p.is;
  g.zs = p.zs;
  g.A = p.A;
  g.dt_bias = p.dt_bias;
  g.in_bias = p.in_bias;
  g.reset = p.reset;
  g.h0 = p.h0;
  g.out = p.out;
  g.h_last = p.h_last;
  g.out_bf16 = p.out_bf16;
  if (q.bytes) {
    char* ws = static_cast<char*>(workspace);
    g.P = reinterpret_cast<float*>(ws + q.off_P);
    g.H = reinterpret_cast<float*>(ws + q.off_H);
    g.G = reinterpret_cast<float*>(ws + q.off_G);
    g.starts = reinterpret_cast<float*>(ws + q.off_starts);
    g.ends = reinterpret_cast<float*>(ws + q.off_ends);
    g.part = reinterpret_cast<float*>(ws + q.off_part);
  }
  g.dout = p.dout;
  g.dh_last = p.dh_last;
  g.du = p.du;
  g.d_dt = p.d_dt;
  g.d_in = p.d_in;
  g.dz = p.dz;
  g.dh0 = p.dh0;
  return g;
}

bool glr_grids_fit(int64_t B, int64_t D, const GlrPieces& p) {
  const int64_t tiles = (D + kLanes - 1) / kLanes;
  return p.pieces <= 0x7fffffff && fits_launch(B * p.pieces * tiles, p.waves * kLanes) &&
         fits_launch(B * tiles * p.ways, kFoldWaves * kLanes);
}

hipError_t launch_glr_aggregates(const GlrPlan& plan, const GlrArgs& g, int64_t count, bool backward,
                                 hipStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(plan.B * count * g.tiles);
  SSM_LOG("launch glr_aggregate: %lld pieces; grid %u x %d threads", static_cast<long long>(count), blocks,
          (backward ? kGlrBwdWaves : kAggWaves) * kLanes);
  return glr_pick<Aggregate>(plan, blocks, g, static_cast<int>(count), backward, stream);
}

hipError_t launch_glr_fold(const GlrPlan& plan, const GlrArgs& g, int64_t count, bool backward, hipStream_t stream) {
  const int ways = backward ? 2 : 1;
  const unsigned blocks = static_cast<unsigned>(plan.B * g.tiles * ways);
  SSM_LOG("launch glr_fold: %lld pieces, %d ways; grid %u x %d threads", static_cast<long long>(count), ways, blocks,
          kFoldWaves * kLanes);
  hipLaunchKernelGGL(glr_fold, dim3(blocks), dim3(kFoldWaves * kLanes), 0, stream, g, count, ways);
  return hipGetLastError();
}

}  // namespace ssm
