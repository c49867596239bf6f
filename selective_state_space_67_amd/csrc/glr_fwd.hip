// The gated linear recurrence forward: the walk over a sequence, the decode
// window, and when to take which (calls with few batch rows and channels go
// through glr_chain.hip).
//
// The walk. A workgroup owns 64 channels and goes through its rows in tiles of
// W K: each of its W waves takes K consecutive rows, works out their decays and
// inputs, and runs the recurrence over them from zero, which leaves the pair
// (P, H) of what the K rows do to an entering state. The pairs meet in LDS; every
// wave folds all W of them, so each knows the state that enters its own rows and
// the one that the tile leaves, and runs its rows once more from the right state.
// One barrier a tile; the next tile's rows are loaded meanwhile. An element is
// read once and written once. What bounds it is the tile's chain of dependent steps
// (decays, recurrence, barrier, fold, recurrence) on the CUs that have a workgroup:
// 64 channels go 30 ns a row, 8 x 2048 x 2048 channels (256 workgroups) 69 us, 3.9 of
// the 5.2 TB/s of a large copy; 1 x 37 x 1536 4.7 us.
#include "glr_device.h"
#include "glr_launch.h"

namespace ssm {
namespace {

constexpr int kWaves = 8, kRows = 8, kTile = kWaves * kRows;

// Rows of the four inputs, K a wave.
template <typename InT, bool IN, bool Z, int K>
struct Rows {
  uint32_t u[K], dt[K], in[K], z[K], reset;
  __device__ __forceinline__ void load(const GlrArgs& g, int64_t row0, int t, int end, int lane, uint32_t at) {
    // a wave whose rows are all past the end reads the last row
    const int64_t row = row0 + min(t, end - 1);
    const int rows = max(1, min(end - t, K));
    load_rows<InT, K>(g.dt, row, g.ds, rows, at, dt);
    if (IN) load_rows<InT, K>(g.in, row, g.is, rows, at, in);
    load_rows<InT, K>(g.u, row, g.us, rows, at, u);
    if (Z) load_rows<InT, K>(g.z, row, g.zs, rows, at, z);
    reset = reset_byte<K>(g.reset, row, t < end ? rows : 0, lane);
  }
  // which of the rows start a document
  __device__ __forceinline__ uint32_t cuts() const {
    return static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(reset != 0));
  }
};

template <typename InT, int DECAY, int MIX, bool IN, bool Z, int W, int K>
__global__ __launch_bounds__(kLanes * W) void glr_walk(const GlrArgs g) {
  __shared__ float2 pairs[2][W][kLanes];
  const int lane = threadIdx.x % kLanes, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int tile = blockIdx.x % g.tiles, batch = blockIdx.x / g.tiles;
  const int channel = tile * kLanes + lane, ch = min(channel, g.D - 1);
  const bool on = channel < g.D;
  const uint32_t at = static_cast<uint32_t>(ch) * sizeof(InT);
  const int64_t state = static_cast<int64_t>(batch) * g.D + ch, row0 = batch * g.L;
  const int end = static_cast<int>(g.L);  // rows are counted in 32 bits (L < 2^27)
  Channel<DECAY> c(g, ch);
  float h = g.h0 ? g.h0[state] : 0.0f;
  Rows<InT, IN, Z, K> x;
  x.load(g, row0, w * K, end, lane, at);
  arrived(h);
  arrived(c.A);
  arrived(c.dt);
  arrived(c.in);
  int buf = 0;
  for (int t0 = 0; t0 < end; t0 += W * K, buf ^= 1) {
    const int t = t0 + w * K;
    const int rows = max(0, min(K, end - t));
    const uint32_t cuts = x.cuts();
    float a[K], b[K], gate[K];
    terms<InT, DECAY, MIX, IN, K>(c, x.u, x.dt, x.in, cuts, a, b);
    if (Z) {
#pragma unroll
      for (int k = 0; k < K; ++k) gate[k] = silu_f32(widen<InT>(x.z[k]));
    }
    if (t0 + W * K < end) x.load(g, row0, t + W * K, end, lane, at);
    if (rows < K) {  // rows past the end do nothing
      keep_branch();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        a[k] = k < rows ? a[k] : 1.0f;
        b[k] = k < rows ? b[k] : 0.0f;
      }
    }
    float P = 1.0f, H = 0.0f, none = 0.0f;
    bool cut = false;
    if (cuts)
      run_rows<false, false, K>(a, b, b, K, cuts, P, H, none, cut);
    else
      run_rows<true, false, K>(a, b, b, K, 0, P, H, none, cut);
    pairs[buf][w][lane] = make_float2(cut ? kCut : P, H);
    __syncthreads();
    float mine = h;
    if (g.reset) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float2 p = pairs[buf][i][lane];
        mine = i == w ? h : mine;
        h = through(p.x, p.y, h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float2 p = pairs[buf][i][lane];
        mine = i == w ? h : mine;
        h = __builtin_fmaf(p.x, h, p.y);
      }
    }
    if (cuts) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        mine = (cuts >> k) & 1 ? b[k] : __builtin_fmaf(a[k], mine, b[k]);
        b[k] = mine;
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        mine = __builtin_fmaf(a[k], mine, b[k]);
        b[k] = mine;
      }
    }
    if (Z) {
#pragma unroll
      for (int k = 0; k < K; ++k) b[k] *= gate[k];
    }
    if (on && rows > 0) store_rows<false, K>(g.out, row0 + t, g.D, rows, ch, g.out_bf16, b);
  }
  if (g.h_last && w == 0 && on) g.h_last[state] = h;
}

// One thread a channel, token by token; the next tokens are loaded ahead, K at a time.
// Bound by the latency of a load, the gates and a store: 2.9 us for 1 x 1536 channels,
// 3.3 for 64 x 2048, whose call takes 8.8 us on the host.
template <typename InT, int DECAY, int MIX, bool IN, bool Z, int K>
__global__ __launch_bounds__(kLanes) void glr_steps(const GlrArgs g) {
  const int lane = threadIdx.x;
  const int tile = blockIdx.x % g.tiles, batch = blockIdx.x / g.tiles;
  const int channel = tile * kLanes + lane, ch = min(channel, g.D - 1);
  const bool on = channel < g.D;
  const uint32_t at = static_cast<uint32_t>(ch) * sizeof(InT);
  const int64_t state = static_cast<int64_t>(batch) * g.D + ch, row0 = batch * g.L;
  Rows<InT, IN, Z, K> x;
  const int L = static_cast<int>(g.L);
  x.load(g, row0, 0, L, lane, at);
  const Channel<DECAY> c(g, ch);
  float h = g.h0 ? g.h0[state] : 0.0f;
  for (int t = 0; t < L; t += K) {
    const uint32_t cuts = x.cuts();
    const int rows = min(K, L - t);
    float a[K], b[K], gate[K];
    terms<InT, DECAY, MIX, IN, K>(c, x.u, x.dt, x.in, cuts, a, b);
    if (Z) {
#pragma unroll
      for (int k = 0; k < K; ++k) gate[k] = silu_f32(widen<InT>(x.z[k]));
    }
    if (t + K < L) x.load(g, row0, t + K, L, lane, at);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < rows) {
        h = (cuts >> k) & 1 ? b[k] : __builtin_fmaf(a[k], h, b[k]);
        b[k] = Z ? h * gate[k] : h;
      }
    if (on) store_rows<false, K>(g.out, row0 + t, g.D, rows, ch, g.out_bf16, b);
  }
  if (g.h_last && on) g.h_last[state] = h;
}

// Up to 256 workgroups, one on a CU, take 16 rows a wave: with half the barriers and folds an
// element their waves wait less (8 x 2048 x 1536 channels, 192 workgroups: 65 us, with 8 rows 71;
// with 16 waves of 16 rows 63). More of them take 8 (of the sequences that long, plan_glr leaves
// the walk those of more than 400 workgroups), and so does what 8 rows a wave cover in a few
// tiles: 1 x 37 x 1536 4.8 us, with 16 rows 6.7.
bool wide_tiles(int64_t blocks, int64_t rows) { return blocks <= 256 && rows >= 8 * kTile; }

struct Walk {
  template <typename InT, int DECAY, int MIX, bool IN, bool Z>
  static hipError_t run(const GlrPlan& plan, const GlrArgs& g, hipStream_t stream) {
    const int64_t blocks = plan.B * g.tiles;
    const bool wide = wide_tiles(blocks, g.L);
    SSM_LOG("launch glr_walk<%d waves of %d rows>: grid %lld x %d threads", kWaves, wide ? 2 * kRows : kRows,
            static_cast<long long>(blocks), kWaves * kLanes);
    const dim3 grid(static_cast<unsigned>(blocks)), block(kWaves * kLanes);
    if (wide)
      hipLaunchKernelGGL((glr_walk<InT, DECAY, MIX, IN, Z, kWaves, 2 * kRows>), grid, block, 0, stream, g);
    else
      hipLaunchKernelGGL((glr_walk<InT, DECAY, MIX, IN, Z, kWaves, kRows>), grid, block, 0, stream, g);
    return hipGetLastError();
  }
};

struct Steps {
  template <typename InT, int DECAY, int MIX, bool IN, bool Z>
  static hipError_t run(unsigned blocks, const GlrArgs& g, hipStream_t stream) {
    if (g.L == 1)
      hipLaunchKernelGGL((glr_steps<InT, DECAY, MIX, IN, Z, 1>), dim3(blocks), dim3(kLanes), 0, stream, g);
    else
      hipLaunchKernelGGL((glr_steps<InT, DECAY, MIX, IN, Z, 4>), dim3(blocks), dim3(kLanes), 0, stream, g);
    return hipGetLastError();
  }
};

int64_t tiles_of(int64_t D) { return (D + kLanes - 1) / kLanes; }

}  // namespace

// Sequences of up to 8 steps have no use for a workgroup's other rows.
bool glr_by_steps(int64_t L) { return L <= 8; }

bool glr_steps_fit(int64_t B, int64_t D) { return fits_launch(B * tiles_of(D), kLanes); }

// The walk gives 64 channels of a batch row to one workgroup, in rounds of one for every CU: 30 ns a
// row and round, however little of the chip a round fills. The chain fills it whatever the shape
// is (0.119 ns a row and 64 channels), but has some 5 us more that do not depend on the shape: a clearing
// launch, tickets, looks. It is taken where the two figures are 7 us apart. us of walk and chain by
// themselves (the launches of a graph; bfloat16, sigmoid gates): 1 x 256 x 256 channels 10.0 and 7.7,
// 1 x 2048 x 1536 57 and 13.6, 2 x 4096 x 2048 118 and 43; 8 x 512 x 1536 17.6 and 18.9, 8 x 1024 x 1536
// 31.5 and 28.7, 8 x 2048 x 1536 65 and 57; 8 x 2048 x 2048 (256 workgroups) 70 and 72; 16 x 2048 x 1280
// (320) 121 and 87; 16 x 1024 x 2048 (512) 67 and 73. Up to some 400 rows the host is slower than either
// where one call follows another, and the chain with its workspace takes it 4 us more: 1 x 256 x 256 12.1
// and 16.8 us a call, 1 x 400 x 256 16.1 and 16.3; a call that is waited for 28.3 and 28.4, 34.5 and 28.9.
GlrPieces plan_glr(int64_t B, int64_t L, int64_t D) {
  const int64_t groups = B * tiles_of(D), rounds = (groups + 255) / 256;
  if (groups < int64_t{1} << 22 && (30000 * rounds - 119 * groups) * L >= 7000000) {
    const GlrPieces chain = plan_glr_chain(B, L, D);
    if (glr_grids_fit(B, D, chain)) return chain;  // (of very many rows of few channels it may need too large a launch)
  }
  GlrPieces p{};
  p.pieces = 1;
  p.rows = L;
  p.waves = kWaves;
  return p;
}

hipError_t launch_glr(const GlrPlan& plan, const GlrPieces& pieces, void* workspace, hipStream_t stream) {
  if (pieces.pieces > 1) return launch_glr_chain(plan, pieces, workspace, stream);
  return glr_pick<Walk>(plan, plan, glr_args(plan), stream);
}

hipError_t launch_glr_steps(const GlrPlan& plan, hipStream_t stream) {
  const GlrArgs g = glr_args(plan);
  const unsigned blocks = static_cast<unsigned>(plan.B * g.tiles);
  SSM_LOG("launch glr_steps: grid %u x %d threads", blocks, kLanes);
  return glr_pick<Steps>(plan, blocks, g, stream);
}

GlrArgs glr_args(const GlrPlan& p) {
  GlrArgs g{};
  g.L = p.L;
  g.D = static_cast<int>(p.D);
  g.tiles = static_cast<int>(tiles_of(p.D));
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
  g.dout = p.dout;
  g.dh_last = p.dh_last;
  g.du = p.du;
  g.d_dt = p.d_dt;
  g.d_in = p.d_in;
  g.dz = p.dz;
  g.dh0 = p.dh0;
  return g;
}

}  // namespace ssm
