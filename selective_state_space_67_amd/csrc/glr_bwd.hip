// Gradients of the gated linear recurrence.
//
// With lam_t the adjoint of h_t,
//
//   dy = dout silu(z),  lam_t = dy_t + a_{t+1} lam_{t+1},  dz = dout h silu'(z)
//   du = lam c i,  d in_raw = lam c u i (1 - i)
//   dg = lam a (h_{t-1} + i u dc/da),  dc/da = -a/c, -1 or 0
//   d dt_raw = dg A s',  dA = sum dg s,  dh0 = a_0 lam_0
//
// and dg = 0 at a reset, which hands no adjoint on either.
//
// Three passes: what every piece of 32 rows does to a state and to an adjoint
// (glr_aggregate: u, dt_raw, in_raw, z, dout read once), the states and adjoints
// that enter the pieces (glr_fold), and here the pieces' gradients, all in
// parallel: a workgroup takes one piece of 64 channels, its waves 8 rows each,
// kept in registers. Each wave's rows act on a state as (P, H) and on an adjoint
// as (P, G); the waves exchange them through LDS once. The parameters' gradients
// are summed over a wave's rows in registers, over the waves in LDS, and over the
// pieces by row_sums, always in the same order.
//
// Bound by memory, the vector ALU close behind: 8 x 2048 x 1536 channels 73 to 79 us for 352 MB
// (4.5 to 4.8 TB/s), 70 vector instructions an element, the ALU busy for 64% of the time. Two passes over the inputs are the price of a
// state that comes from the front and an adjoint that comes from behind. With a first pass
// for the adjoints alone and this one getting its states from a chain of workgroups (as in
// glr_chain.hip), u and in_raw are read only once, but this pass then waits: 29 and 95 us
// in place of 49 and 73, and few columns wait longest (1 x 131072 x 256: 289 us in place
// of 258).
#include <type_traits>

#include "glr_device.h"
#include "glr_launch.h"
#include "kernels_block.h"

namespace ssm {
namespace {

constexpr int kRows = 8, kPiece = kGlrBwdWaves * kRows;

template <typename InT, int DECAY, int MIX, bool IN, bool Z, int W, int K>
__global__ __launch_bounds__(kLanes * W) void glr_grads(const GlrArgs g) {
  __shared__ float ex[3][W][kLanes];  // P, H, G; then the three sums
  const int lane = threadIdx.x % kLanes, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  // the pieces that were read last come first: some of them are in the last-level cache still
  const int block = gridDim.x - 1 - blockIdx.x;
  const int tile = block % g.tiles, rest = block / g.tiles;
  const int piece = rest % g.pieces, batch = rest / g.pieces;
  const int channel = tile * kLanes + lane, ch = min(channel, g.D - 1);
  const bool on = channel < g.D;
  const uint32_t at = static_cast<uint32_t>(ch) * sizeof(InT);
  const int64_t row0 = batch * g.L, t = static_cast<int64_t>(piece) * (W * K) + w * K;
  const int rows = static_cast<int>(max(int64_t{0}, min(int64_t{K}, g.L - t)));
  const int64_t row = row0 + min(t, g.L - 1);
  const int have = max(rows, 1);
  uint32_t ru[K], rdt[K], rin[K], rz[K], rdy[K];
  load_rows<InT, K>(g.dt, row, g.ds, have, at, rdt);
  if (IN) load_rows<InT, K>(g.in, row, g.is, have, at, rin);
  load_rows<InT, K>(g.u, row, g.us, have, at, ru);
  load_rows<InT, K>(g.dout, row, g.D, have, at, rdy);
  if (Z) load_rows<InT, K>(g.z, row, g.zs, have, at, rz);
  const uint32_t reset = reset_byte<K>(g.reset, row, rows, lane);
  const int64_t joint = (static_cast<int64_t>(batch) * g.pieces + piece) * g.D + ch;
  float h = g.starts[joint], m = g.ends[joint];
  const Channel<DECAY> chn(g, ch);
  const uint32_t cuts = static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(reset != 0));

  float a[K], c[K], s[K], e[K], dy[K], b[K];  // b = c i u
  decays<InT, DECAY, MIX, K>(chn, rdt, s, e, a, c);
  // s' = s (1 - s). Of the two factors the smaller one is kept, which gives the other one and the
  // product to full precision: s up to 1/2, else 1 - s with its sign turned.
  if (DECAY == kGlrSigmoid) {
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = s[k] > 0.5f ? -(e[k] * s[k]) : s[k];
  }
  const bool plain = rows == K && cuts == 0;
  if (cuts) {
    keep_branch();
#pragma unroll
    for (int k = 0; k < K; ++k)
      if ((cuts >> k) & 1) c[k] = 1.0f;
  }
  // what the adjoint is multiplied by: c i for du, b (1 - i) for d in_raw, A s' for d dt_raw, and i u dc/da
  float ci[K], in_slope[K], xdc[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float x = widen<InT>(ru[k]), i_rest = 0.0f;
    ci[k] = c[k];
    if (IN) {
      const Sigmoid i(__builtin_fmaf(widen<InT>(rin[k]), -kLog2e, chn.in));
      i_rest = fminf(i.e, 3.4e38f) * i.value;
      x *= i.value;
      ci[k] = MIX == kGlrOne ? i.value : c[k] * i.value;
    }
    b[k] = MIX == kGlrOne ? x : c[k] * x;
    if (IN) in_slope[k] = b[k] * i_rest;
    // where a rounds to 1, c is 0 and its slope infinite, but what the gate and A get tends to 0
    if (MIX == kGlrUnit) xdc[k] = c[k] == 0.0f ? 0.0f : -a[k] * fast_rcp(c[k]) * x;
    if (MIX == kGlrRest) xdc[k] = -x;
    dy[k] = Z ? widen<InT>(rdy[k]) * silu_f32(widen<InT>(rz[k])) : widen<InT>(rdy[k]);
  }
  float P = 1.0f, H = 0.0f, G = 0.0f;
  bool cut = false;
  if (plain)
    run_rows<true, true, K>(a, b, dy, K, 0, P, H, G, cut);
  else
    run_rows<false, true, K>(a, b, dy, rows, cuts, P, H, G, cut);
  ex[0][w][lane] = cut ? kCut : P;
  ex[1][w][lane] = H;
  ex[2][w][lane] = G;
  __syncthreads();
  for (int j = 0; j < w; ++j) h = through(ex[0][j][lane], ex[1][j][lane], h);
  for (int j = W - 1; j > w; --j) m = through(ex[0][j][lane], ex[2][j][lane], m);

  float sum_A = 0.0f, sum_dt = 0.0f, sum_in = 0.0f;
  auto gradients = [&](auto all) {
    constexpr bool PLAIN = decltype(all)::value;
    float before[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      before[k] = h;
      h = !PLAIN && ((cuts >> k) & 1) ? b[k] : __builtin_fmaf(a[k], h, b[k]);
      if (Z) {  // b becomes dz
        const float z = widen<InT>(rz[k]), sz = sigmoid_f32(z);
        b[k] = widen<InT>(rdy[k]) * h * sz * __builtin_fmaf(z, 1.0f - sz, 1.0f);
      }
    }
    if (Z && on) store_rows<PLAIN, K>(g.dz, row, g.D, rows, ch, g.out_bf16, b);
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      if (!PLAIN && k >= rows) continue;
      const float lam = dy[k] + m;
      b[k] = lam * ci[k];  // du
      if (IN) {
        in_slope[k] *= lam;  // d in_raw
        sum_in += in_slope[k];
      }
      if (!PLAIN && ((cuts >> k) & 1)) {
        m = dy[k] = 0.0f;
        continue;
      }
      m = a[k] * lam;
      const float dg = m * (MIX == kGlrOne ? before[k] : before[k] + xdc[k]);
      float gate = s[k], slope;
      if (DECAY == kGlrSigmoid) {
        gate = __float_as_int(s[k]) < 0 ? 1.0f + s[k] : s[k];
        slope = __builtin_fmaf(-fabsf(s[k]), fabsf(s[k]), fabsf(s[k]));
      } else {
        slope = sigmoid_f32(widen<InT>(rdt[k]) + chn.dt);
      }
      sum_A = __builtin_fmaf(dg, gate, sum_A);
      dy[k] = dg * chn.A * slope;  // d dt_raw
      sum_dt += dy[k];
    }
    if (on) {
      store_rows<PLAIN, K>(g.du, row, g.D, rows, ch, g.out_bf16, b);
      if (IN) store_rows<PLAIN, K>(g.d_in, row, g.D, rows, ch, g.out_bf16, in_slope);
      store_rows<PLAIN, K>(g.d_dt, row, g.D, rows, ch, g.out_bf16, dy);
    }
  };
  if (plain)
    gradients(std::true_type{});
  else if (rows > 0)
    gradients(std::false_type{});
  __syncthreads();
  ex[0][w][lane] = sum_A;
  ex[1][w][lane] = sum_dt;
  ex[2][w][lane] = sum_in;
  __syncthreads();
  if (w < 3 && on) {
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) v += ex[w][j][lane];
    g.part[((static_cast<int64_t>(batch) * g.pieces + piece) * 3 + w) * g.D + ch] = v;
  }
}

struct Grads {
  template <typename InT, int DECAY, int MIX, bool IN, bool Z>
  static hipError_t run(unsigned blocks, const GlrArgs& g, hipStream_t stream) {
    hipLaunchKernelGGL((glr_grads<InT, DECAY, MIX, IN, Z, kGlrBwdWaves, kRows>), dim3(blocks), dim3(kGlrBwdWaves * kLanes), 0,
                       stream, g);
    return hipGetLastError();
  }
};

}  // namespace

GlrPieces plan_glr_bwd(int64_t B, int64_t L, int64_t D) {
  GlrPieces p{};
  p.rows = kPiece;
  p.waves = kGlrBwdWaves;
  p.pieces = (L + kPiece - 1) / kPiece;
  const size_t each = (static_cast<size_t>(B) * p.pieces * D * sizeof(float) + 255) / 256 * 256;
  p.off_H = each;
  p.off_G = 2 * each;
  p.off_starts = 3 * each;
  p.off_ends = 4 * each;
  p.off_part = 5 * each;
  p.off_segments = 8 * each;
  p.bytes = p.off_segments;
  p.segments = 1;
  p.each = static_cast<int>(p.pieces);
  // Few columns and many pieces: the fold in segments. us of one fold and of the three launches in
  // segments, which start some 3 us later: 4 columns 15.6 and 12.5 with 767 and 768 pieces, 88 and 17.6
  // with 4096; 128 columns, whose one fold reaches every CU, 24 and 52 with 512.
  if (p.pieces >= 768 && B * ((D + kLanes - 1) / kLanes) < 64) {
    p.each = kGlrSegment;
    p.segments = (p.pieces + kGlrSegment - 1) / kGlrSegment;
    p.bytes += (5 * static_cast<size_t>(B) * p.segments * D * sizeof(float) + 255) / 256 * 256;
  }
  return p;
}

hipError_t launch_glr_bwd(const GlrPlan& plan, const GlrPieces& pieces, void* workspace, hipStream_t stream) {
  GlrArgs g = glr_args(plan);
  char* ws = static_cast<char*>(workspace);
  g.pieces = static_cast<int>(pieces.pieces);
  g.P = reinterpret_cast<float*>(ws + pieces.off_P);
  g.H = reinterpret_cast<float*>(ws + pieces.off_H);
  g.G = reinterpret_cast<float*>(ws + pieces.off_G);
  g.starts = reinterpret_cast<float*>(ws + pieces.off_starts);
  g.ends = reinterpret_cast<float*>(ws + pieces.off_ends);
  g.part = reinterpret_cast<float*>(ws + pieces.off_part);
  hipError_t e = launch_glr_aggregates(plan, g, stream);
  if (e == hipSuccess) e = launch_glr_fold(plan, g, pieces, reinterpret_cast<float*>(ws + pieces.off_segments), stream);
  if (e != hipSuccess) return e;
  const unsigned blocks = static_cast<unsigned>(plan.B * pieces.pieces * g.tiles);
  SSM_LOG("launch glr_grads: %lld pieces of %d rows; grid %u x %d threads", static_cast<long long>(pieces.pieces),
          kPiece, blocks, kGlrBwdWaves * kLanes);
  e = glr_pick<Grads>(plan, blocks, g, stream);
  if (e != hipSuccess) return e;
  // (dim <= 2^24: below 2^32 threads)
  const int64_t sums = plan.B * pieces.pieces;
  return launch_row_sums(g.part, 3 * plan.D, g.D,
                         {{plan.dA, 0, sums, 1}, {plan.d_dt_bias, plan.D, sums, 1}, {plan.din_bias, 2 * plan.D, sums, 1}},
                         stream);
}

}  // namespace ssm
