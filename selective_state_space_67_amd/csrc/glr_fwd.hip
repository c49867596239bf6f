// The gated linear recurrence forward: the walk over a sequence (or over one
// piece of it), and the decode window.
//
// The walk. A workgroup owns 64 channels and goes through its rows in tiles of
// W K: each of its W waves takes K consecutive rows, works out their decays and
// inputs, and runs the recurrence over them from zero, which leaves the pair
// (P, H) of what the K rows do to an entering state. The pairs meet in LDS; every
// wave folds all W of them, so each knows the state that enters its own rows and
// the one that the tile leaves, and runs its rows once more from the right state.
// One barrier a tile; the next tile's rows are loaded meanwhile. An element is
// read once and written once.
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
  const int tile = blockIdx.x % g.tiles, rest = blockIdx.x / g.tiles;
  const int piece = rest % g.pieces, batch = rest / g.pieces;
  const int channel = tile * kLanes + lane, ch = min(channel, g.D - 1);
  const bool on = channel < g.D;
  const uint32_t at = static_cast<uint32_t>(ch) * sizeof(InT);
  const int64_t state = static_cast<int64_t>(batch) * g.D + ch, row0 = batch * g.L;
  // rows are counted in 32 bits (L < 2^27)
  const int begin = static_cast<int>(piece * g.piece_rows);
  const int end = static_cast<int>(min(g.L, begin + g.piece_rows));
  Channel<DECAY> c(g, ch);
  float h = g.pieces > 1 ? g.starts[(static_cast<int64_t>(batch) * g.pieces + piece) * g.D + ch]
            : g.h0       ? g.h0[state]
                         : 0.0f;
  Rows<InT, IN, Z, K> x;
  x.load(g, row0, begin + w * K, end, lane, at);
  arrived(h);
  arrived(c.A);
  arrived(c.dt);
  arrived(c.in);
  int buf = 0;
  for (int t0 = begin; t0 < end; t0 += W * K, buf ^= 1) {
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
  if (g.h_last && piece == g.pieces - 1 && w == 0 && on) g.h_last[state] = h;
}

// One thread a channel, token by token; the next tokens are loaded ahead, K at a time.
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

// Few workgroups, none of which shares its CU with another, take 16 rows a wave: with half the
// barriers and folds an element their waves wait less (8 x 2048 x 1536 channels, 192 workgroups:
// 65 us, with 8 rows 71; with 16 waves of 16 rows 63). Many take 8: 1 x 131072 x 256 in 512
// pieces 58 us, with 16 rows 63, with 16 waves 81. So does what 8 rows a wave cover in a few tiles:
// 1 x 37 x 1536 4.8 us, with 16 rows 6.7.
bool wide_tiles(int64_t blocks, int64_t rows) { return blocks <= 384 && rows >= 8 * kTile; }

struct Walk {
  template <typename InT, int DECAY, int MIX, bool IN, bool Z>
  static hipError_t run(const GlrPlan& plan, const GlrArgs& g, hipStream_t stream) {
    const int64_t blocks = plan.B * g.pieces * g.tiles;
    const bool wide = wide_tiles(blocks, g.piece_rows);
    SSM_LOG("launch glr_walk<%d waves of %d rows>: %d pieces of %lld rows; grid %lld x %d threads", kWaves,
            wide ? 2 * kRows : kRows, g.pieces, static_cast<long long>(g.piece_rows), static_cast<long long>(blocks),
            kWaves * kLanes);
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

GlrPieces plan_glr(int64_t B, int64_t L, int64_t D, int requested) {
  GlrPieces p{};
  const int64_t tiles = (L + kTile - 1) / kTile, groups = B * tiles_of(D);
  int64_t pieces = 1;
  if (requested > 0)
    pieces = requested;
  else if (groups < 128 && tiles >= 8)
    pieces = 1024 / groups;
  pieces = pieces < tiles ? pieces : tiles;
  if (pieces < 1) pieces = 1;
  p.rows = (tiles + pieces - 1) / pieces * kTile;
  p.pieces = (L + p.rows - 1) / p.rows;
  p.waves = kWaves;
  p.ways = p.pieces > 1 ? 1 : 0;
  if (p.pieces > 1) {
    const size_t each = (static_cast<size_t>(B) * p.pieces * D * sizeof(float) + 255) / 256 * 256;
    p.off_P = 0;
    p.off_H = each;
    p.off_starts = 2 * each;
    p.bytes = 3 * each;
  }
  return p;
}

hipError_t launch_glr(const GlrPlan& plan, const GlrPieces& pieces, void* workspace, hipStream_t stream) {
  const GlrArgs g = glr_args(plan, pieces, workspace);
  if (pieces.pieces > 1) {
    hipError_t e = launch_glr_aggregates(plan, g, pieces.pieces - 1, false, stream);
    if (e == hipSuccess) e = launch_glr_fold(plan, g, pieces.pieces - 1, false, stream);
    if (e != hipSuccess) return e;
  }
  return glr_pick<Walk>(plan, plan, g, stream);
}

hipError_t launch_glr_steps(const GlrPlan& plan, hipStream_t stream) {
  GlrPieces one{};
  one.pieces = 1;
  one.rows = plan.L;
  const GlrArgs g = glr_args(plan, one, nullptr);
  const unsigned blocks = static_cast<unsigned>(plan.B * g.tiles);
  SSM_LOG("launch glr_steps: grid %u x %d threads", blocks, kLanes);
  return glr_pick<Steps>(plan, blocks, g, stream);
}

}  // namespace ssm
