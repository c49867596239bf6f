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

constexpr int kWaves = 16, kRows = 8, kTile = kWaves * kRows;

template <typename InT, int K>
struct Rows {
  uint32_t u[K], dt[K], in[K], z[K], reset;
  __device__ __forceinline__ void load(const GlrArgs& g, int64_t row0, int64_t t, int64_t end, int lane, uint32_t at) {
    // a wave whose rows are all past the end reads the last row
    const int64_t row = row0 + (t < end ? t : end - 1);
    const int rows = t < end ? static_cast<int>(end - t < K ? end - t : K) : 1;
    load_rows<InT, K>(g.u, row, g.us, rows, at, u);
    load_rows<InT, K>(g.dt, row, g.ds, rows, at, dt);
    if (g.in) load_rows<InT, K>(g.in, row, g.is, rows, at, in);
    if (g.z) load_rows<InT, K>(g.z, row, g.zs, rows, at, z);
    reset = reset_byte<K>(g.reset, row, t < end ? rows : 0, lane);
  }
};

// A channel's constants.
struct Channel {
  float A, dt_bias, in_bias;
  __device__ __forceinline__ Channel(const GlrArgs& g, int ch)
      : A(g.A[ch]), dt_bias(g.dt_bias ? g.dt_bias[ch] : 0.0f), in_bias(g.in_bias ? g.in_bias[ch] : 0.0f) {}
};

// Decays a and inputs b of K rows; cuts: the rows that start a document.
template <typename InT, int DECAY, int MIX, int K>
__device__ __forceinline__ void terms(const GlrArgs& g, const Channel& c, const Rows<InT, K>& x, uint32_t cuts,
                                      float (&a)[K], float (&b)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) b[k] = widen<InT>(x.u[k]);
  if (g.in) {
#pragma unroll
    for (int k = 0; k < K; ++k) b[k] *= sigmoid_f32(widen<InT>(x.in[k]) + c.in_bias);
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float m;
    decay_terms<MIX>(c.A * decay_gate<DECAY>(widen<InT>(x.dt[k]) + c.dt_bias), a[k], m);
    if (MIX != kGlrOne) b[k] *= (cuts >> k) & 1 ? 1.0f : m;
  }
}

template <int K, bool CUTS>
__device__ __forceinline__ void run_rows(const float (&a)[K], const float (&b)[K], uint32_t cuts, float& P, float& H) {
  P = 1.0f;
  H = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    P *= a[k];
    H = CUTS && ((cuts >> k) & 1) ? b[k] : __builtin_fmaf(a[k], H, b[k]);
  }
  if (CUTS) P = kCut;
}

template <typename InT, int DECAY, int MIX, int W, int K>
__global__ __launch_bounds__(kLanes * W) void glr_walk(const GlrArgs g) {
  __shared__ float2 pairs[2][W][kLanes];
  const int lane = threadIdx.x % kLanes, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int tile = blockIdx.x % g.tiles, rest = blockIdx.x / g.tiles;
  const int piece = rest % g.pieces, batch = rest / g.pieces;
  const int channel = tile * kLanes + lane, ch = min(channel, g.D - 1);
  const bool on = channel < g.D;
  const uint32_t at = static_cast<uint32_t>(ch) * sizeof(InT);
  const Channel c(g, ch);
  const int64_t state = static_cast<int64_t>(batch) * g.D + ch, row0 = batch * g.L;
  float h = g.pieces > 1 ? g.starts[(static_cast<int64_t>(batch) * g.pieces + piece) * g.D + ch]
            : g.h0       ? g.h0[state]
                         : 0.0f;
  const int64_t begin = piece * g.piece_rows, end = min(g.L, begin + g.piece_rows);
  const int out_size = g.out_bf16 ? 2 : 4;
  Rows<InT, K> x;
  x.load(g, row0, begin + w * K, end, lane, at);
  int buf = 0;
  for (int64_t t0 = begin; t0 < end; t0 += W * K, buf ^= 1) {
    const int64_t t = t0 + w * K;
    const int rows = static_cast<int>(max(int64_t{0}, min(int64_t{K}, end - t)));
    const uint32_t cuts = static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(x.reset != 0));
    float a[K], b[K], gate[K];
    terms<InT, DECAY, MIX, K>(g, c, x, cuts, a, b);
    if (g.z) {
#pragma unroll
      for (int k = 0; k < K; ++k) gate[k] = silu_f32(widen<InT>(x.z[k]));
    }
    if (t0 + W * K < end) x.load(g, row0, t + W * K, end, lane, at);
    if (rows < K) {  // rows past the end do nothing
#pragma unroll
      for (int k = 0; k < K; ++k) {
        a[k] = k < rows ? a[k] : 1.0f;
        b[k] = k < rows ? b[k] : 0.0f;
      }
    }
    float P, H;
    if (cuts)
      run_rows<K, true>(a, b, cuts, P, H);
    else
      run_rows<K, false>(a, b, cuts, P, H);
    pairs[buf][w][lane] = make_float2(P, H);
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
    if (g.z) {
#pragma unroll
      for (int k = 0; k < K; ++k) b[k] *= gate[k];
    }
    if (on) {
      char* out = static_cast<char*>(g.out) + (row0 + t) * g.D * out_size;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (k < rows) store_result(out, ch, b[k], g.out_bf16);
        out += static_cast<int64_t>(g.D) * out_size;
      }
    }
  }
  if (g.h_last && piece == g.pieces - 1 && w == 0 && on) g.h_last[state] = h;
}

// One thread a channel, token by token; the next tokens are loaded ahead, K at a time.
template <typename InT, int DECAY, int MIX, int K>
__global__ __launch_bounds__(kLanes) void glr_steps(const GlrArgs g) {
  const int lane = threadIdx.x;
  const int tile = blockIdx.x % g.tiles, batch = blockIdx.x / g.tiles;
  const int channel = tile * kLanes + lane, ch = min(channel, g.D - 1);
  const bool on = channel < g.D;
  const uint32_t at = static_cast<uint32_t>(ch) * sizeof(InT);
  const int64_t state = static_cast<int64_t>(batch) * g.D + ch, row0 = batch * g.L;
  Rows<InT, K> x;
  x.load(g, row0, 0, g.L, lane, at);
  const Channel c(g, ch);
  float h = g.h0 ? g.h0[state] : 0.0f;
  const int out_size = g.out_bf16 ? 2 : 4;
  for (int64_t t = 0; t < g.L; t += K) {
    const uint32_t cuts = static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(x.reset != 0));
    const int rows = static_cast<int>(min(int64_t{K}, g.L - t));
    float a[K], b[K], gate[K];
    terms<InT, DECAY, MIX, K>(g, c, x, cuts, a, b);
    if (g.z) {
#pragma unroll
      for (int k = 0; k < K; ++k) gate[k] = silu_f32(widen<InT>(x.z[k]));
    }
    if (t + K < g.L) x.load(g, row0, t + K, g.L, lane, at);
    char* out = static_cast<char*>(g.out) + (row0 + t) * g.D * out_size;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k < rows) {
        h = (cuts >> k) & 1 ? b[k] : __builtin_fmaf(a[k], h, b[k]);
        if (on) store_result(out, ch, g.z ? h * gate[k] : h, g.out_bf16);
        out += static_cast<int64_t>(g.D) * out_size;
      }
    }
  }
  if (g.h_last && on) g.h_last[state] = h;
}

struct Walk {
  template <typename InT, int DECAY, int MIX>
  static hipError_t run(unsigned blocks, const GlrArgs& g, hipStream_t stream) {
    hipLaunchKernelGGL((glr_walk<InT, DECAY, MIX, kWaves, kRows>), dim3(blocks), dim3(kWaves * kLanes), 0, stream, g);
    return hipGetLastError();
  }
};

struct Steps {
  template <typename InT, int DECAY, int MIX>
  static hipError_t run(unsigned blocks, const GlrArgs& g, hipStream_t stream) {
    if (g.L == 1)
      hipLaunchKernelGGL((glr_steps<InT, DECAY, MIX, 1>), dim3(blocks), dim3(kLanes), 0, stream, g);
    else
      hipLaunchKernelGGL((glr_steps<InT, DECAY, MIX, 4>), dim3(blocks), dim3(kLanes), 0, stream, g);
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
    pieces = 2048 / groups;
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
  const unsigned blocks = static_cast<unsigned>(plan.B * pieces.pieces * g.tiles);
  SSM_LOG("launch glr_walk<%d waves of %d rows>: %lld pieces of %lld rows; grid %u x %d threads", kWaves, kRows,
          static_cast<long long>(pieces.pieces), static_cast<long long>(pieces.rows), blocks, kWaves * kLanes);
  return glr_pick<Walk>(plan, blocks, g, stream);
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
