// The first two passes of the gated linear recurrence's backward: what each piece of
// a sequence does to a state and to an adjoint, and the states and adjoints that enter
// the pieces.
//
// A piece maps the state h that enters it to P h + H, and the adjoint m that enters it
// from behind to P m + G, with P the product of its decays and
//   H = the state it leaves from zero,   G = sum_t (prod_{r <= t} a_r) dout_t silu(z_t)
// A workgroup makes a piece's three values for 64 channels, each of its waves those of
// 8 rows: 8 x 2048 x 1536 channels 48.8 us for 201 MB, 4.1 TB/s. Reading them alone takes
// 37 us (5.5 TB/s) by the same loads of two bytes a lane as by those of 16; the rest is the
// gates and the recurrence on top (278 vector instructions a wave, the ALU busy for half of
// the time), which a workgroup begins when its loads are there, and after which it ends. The fold runs the same scheme over the pieces that the walk runs
// over rows. A workgroup of it gets through 128 pieces in 2.7 us, which is what its CU
// draws from memory; many pieces (plan_glr_bwd) go in segments, first for what each
// segment does, and again once the states and adjoints at its ends are known.
#include "glr_device.h"
#include "glr_launch.h"

namespace ssm {
namespace {

constexpr int kAggRows = 8;
constexpr int kFoldWaves = kGlrSegment / 4;

template <typename InT, int DECAY, int MIX, bool IN, bool Z, int W, int K>
__global__ __launch_bounds__(W * kLanes) void glr_aggregate(const GlrArgs g) {
  __shared__ float ex[3][W][kLanes];
  const int lane = threadIdx.x % kLanes, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int tile = blockIdx.x % g.tiles, rest = blockIdx.x / g.tiles;
  const int piece = rest % g.pieces, batch = rest / g.pieces;
  const int channel = tile * kLanes + lane, ch = min(channel, g.D - 1);
  const uint32_t at = static_cast<uint32_t>(ch) * sizeof(InT);
  const int L = static_cast<int>(g.L), t = piece * (W * K) + w * K;  // (the last piece's waves may have no rows)
  const int rows = max(0, min(K, L - t)), have = max(rows, 1);
  const int64_t row = batch * g.L + min(t, L - 1);
  uint32_t u[K], dt[K], in[K], z[K], rdy[K];
  load_rows<InT, K>(g.dt, row, g.ds, have, at, dt);
  if (IN) load_rows<InT, K>(g.in, row, g.is, have, at, in);
  load_rows<InT, K>(g.u, row, g.us, have, at, u);
  load_rows<InT, K>(g.dout, row, g.D, have, at, rdy);
  if (Z) load_rows<InT, K>(g.z, row, g.zs, have, at, z);
  const uint32_t reset = reset_byte<K>(g.reset, row, rows, lane);
  const Channel<DECAY> c(g, ch);
  const uint32_t cuts = static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(reset != 0));
  float a[K], b[K], dy[K], P = 1.0f, H = 0.0f, G = 0.0f;
  bool cut = false;
  terms<InT, DECAY, MIX, IN, K>(c, u, dt, in, cuts, a, b);
#pragma unroll
  for (int k = 0; k < K; ++k) dy[k] = Z ? widen<InT>(rdy[k]) * silu_f32(widen<InT>(z[k])) : widen<InT>(rdy[k]);
  if (rows == K && cuts == 0)
    run_rows<true, true, K>(a, b, dy, K, 0, P, H, G, cut);
  else
    run_rows<false, true, K>(a, b, dy, rows, cuts, P, H, G, cut);
  ex[0][w][lane] = cut ? kCut : P;
  ex[1][w][lane] = H;
  ex[2][w][lane] = G;
  __syncthreads();
  if (w >= 3 || channel >= g.D) return;
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

// A level of the fold: `count` pieces of a batch row, in segments of `each`.
struct FoldLevel {
  const float* P;  // (B, count, D)
  const float* H;
  const float* G;
  const float* state;    // (B, segments, D): before a segment, null: 0
  const float* adjoint;  // and behind it
  float* starts;         // (B, count, D): before a piece
  float* ends;           // and behind it
  float* sum_P;  // (B, segments, D): what a segment does
  float* sum_H;
  float* sum_G;
  float* dh0;  // what leaves a segment to the front, or null
  int D, tiles, count, each, segments;
};

// States entering a segment's pieces, or (BACK) adjoints entering them from behind, the last
// piece first; or (SUM) what a segment does. A workgroup takes 64 channels of a segment, its waves K
// pieces each.
template <bool BACK, bool SUM, int K>
__device__ __forceinline__ void fold_pieces(const FoldLevel& f, int64_t batch, int segment, int ch, bool on, int lane,
                                            int w, float2 (*pairs)[kFoldWaves][kLanes]) {
  constexpr int W = kFoldWaves;
  const int64_t from = batch * f.count + static_cast<int64_t>(segment) * f.each;  // of all pieces
  const int count = min(f.each, f.count - segment * f.each);
  const int64_t base = (from + (BACK ? count - 1 : 0)) * f.D + ch, step = BACK ? -int64_t{f.D} : int64_t{f.D};
  const int64_t joint = (batch * f.segments + segment) * f.D + ch;
  const float* add = BACK ? f.G : f.H;
  float* to = BACK ? f.ends : f.starts;
  const float* first = BACK ? f.adjoint : f.state;
  float h = !SUM && first ? first[joint] : 0.0f, all = 1.0f;
  int buf = 0;
  for (int i0 = 0; i0 < count; i0 += W * K, buf ^= 1) {
    float a[K], b[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = i0 + w * K + k;
      a[k] = i < count ? f.P[base + i * step] : 1.0f;
      b[k] = i < count ? add[base + i * step] : 0.0f;
    }
    float P = 1.0f, H = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      H = through(a[k], b[k], H);
      P = joined(P, a[k]);
    }
    pairs[buf][w][lane] = make_float2(P, H);
    __syncthreads();
    float mine = h;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 p = pairs[buf][i][lane];
      mine = i == w ? h : mine;
      h = through(p.x, p.y, h);
      if (SUM) all = joined(all, p.x);
    }
    if (!SUM) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int i = i0 + w * K + k;
        if (on && i < count) to[base + i * step] = mine;
        mine = through(a[k], b[k], mine);
      }
    }
  }
  if (w != 0 || !on) return;
  if (SUM) {
    (BACK ? f.sum_G : f.sum_H)[joint] = h;
    if (!BACK) f.sum_P[joint] = all;
  } else if (BACK && f.dh0) {
    f.dh0[joint] = h;
  }
}

template <bool SUM, int K>
__global__ __launch_bounds__(kFoldWaves * kLanes) void glr_fold(const FoldLevel f) {
  __shared__ float2 pairs[2][kFoldWaves][kLanes];
  const int lane = threadIdx.x % kLanes, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int way = blockIdx.x % 2, rest = blockIdx.x / 2;
  const int tile = rest % f.tiles, row = rest / f.tiles;
  const int segment = row % f.segments;
  const int64_t batch = row / f.segments;
  const int channel = tile * kLanes + lane, ch = min(channel, f.D - 1);
  const bool on = channel < f.D;
  if (way == 0)
    fold_pieces<false, SUM, K>(f, batch, segment, ch, on, lane, w, pairs);
  else
    fold_pieces<true, SUM, K>(f, batch, segment, ch, on, lane, w, pairs);
}

// 64 pieces: with 4 a wave 7.5 us, with 8 8.2 (8 x 1536 channels).
template <bool SUM>
hipError_t fold_level(const GlrPlan& plan, const FoldLevel& f, hipStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(plan.B * f.segments * f.tiles * 2);
  SSM_LOG("launch glr_fold: %d pieces in %d segments; grid %u x %d threads", f.count, f.segments, blocks,
          kFoldWaves * kLanes);
  if (SUM || f.each <= kGlrSegment)
    hipLaunchKernelGGL((glr_fold<SUM, 4>), dim3(blocks), dim3(kFoldWaves * kLanes), 0, stream, f);
  else
    hipLaunchKernelGGL((glr_fold<false, 8>), dim3(blocks), dim3(kFoldWaves * kLanes), 0, stream, f);
  return hipGetLastError();
}

struct Aggregate {
  template <typename InT, int DECAY, int MIX, bool IN, bool Z>
  static hipError_t run(unsigned blocks, const GlrArgs& g, hipStream_t stream) {
    hipLaunchKernelGGL((glr_aggregate<InT, DECAY, MIX, IN, Z, kGlrBwdWaves, kAggRows>), dim3(blocks),
                       dim3(kGlrBwdWaves * kLanes), 0, stream, g);
    return hipGetLastError();
  }
};

}  // namespace

bool glr_grids_fit(int64_t B, int64_t D, const GlrPieces& p) {
  const int64_t columns = B * ((D + kLanes - 1) / kLanes);
  const bool folds = p.off_G != 0;  // (the backward's pieces)
  return p.pieces <= 0x7fffffff && fits_launch(columns * p.pieces, p.waves * kLanes) &&
         (!folds || fits_launch(columns * 2 * p.segments, kFoldWaves * kLanes));
}

hipError_t launch_glr_aggregates(const GlrPlan& plan, const GlrArgs& g, hipStream_t stream) {
  const unsigned blocks = static_cast<unsigned>(plan.B * g.pieces * g.tiles);
  SSM_LOG("launch glr_aggregate: %d pieces; grid %u x %d threads", g.pieces, blocks, kGlrBwdWaves * kLanes);
  return glr_pick<Aggregate>(plan, blocks, g, stream);
}

hipError_t launch_glr_fold(const GlrPlan& plan, const GlrArgs& g, const GlrPieces& p, float* segments,
                           hipStream_t stream) {
  FoldLevel all{};
  all.P = g.P;
  all.H = g.H;
  all.G = g.G;
  all.D = g.D;
  all.tiles = g.tiles;
  all.count = g.pieces;
  all.each = p.each;
  all.segments = static_cast<int>(p.segments);
  if (p.segments == 1) {
    all.state = g.h0;
    all.adjoint = g.dh_last;
    all.starts = g.starts;
    all.ends = g.ends;
    all.dh0 = g.dh0;
    return fold_level<false>(plan, all, stream);
  }
  // the segments' sums, what enters the segments, what enters their pieces
  const int64_t size = plan.B * p.segments * plan.D;
  FoldLevel sums = all, joints = all;
  sums.sum_P = segments;
  sums.sum_H = segments + size;
  sums.sum_G = segments + 2 * size;
  joints.P = sums.sum_P;
  joints.H = sums.sum_H;
  joints.G = sums.sum_G;
  joints.state = g.h0;
  joints.adjoint = g.dh_last;
  joints.starts = segments + 3 * size;
  joints.ends = segments + 4 * size;
  joints.dh0 = g.dh0;
  joints.count = joints.each = all.segments;
  joints.segments = 1;
  all.state = joints.starts;
  all.adjoint = joints.ends;
  all.starts = g.starts;
  all.ends = g.ends;
  hipError_t e = fold_level<true>(plan, sums, stream);
  if (e == hipSuccess) e = fold_level<false>(plan, joints, stream);
  return e == hipSuccess ? fold_level<false>(plan, all, stream) : e;
}

}  // namespace ssm
