// The gated linear recurrence forward in one pass over a sequence cut into pieces
// that follow each other on the chip, for calls whose batch rows and channels are
// too few to fill it with one workgroup for each.
//
// A workgroup takes 64 channels and one piece of W K rows, kept in registers. Its
// rows act on the state that enters the piece as h -> P h + H. It publishes that
// pair at once, then gathers the state that enters its piece from what the
// workgroups before it have published, and runs its rows from there. So that no
// state has to pass through every piece, sixteen pieces make a group and sixteen
// groups a range: a group's last workgroup publishes the group's pair, a range's
// last one the state after it, and a piece needs the state that enters its range,
// the pairs of at most fifteen groups and of at most fifteen pieces, always joined
// in that order (repeated calls give identical bits).
//
// Every wait ends. The workgroups of 64 channels take their pieces from a counter of
// these channels, so whoever waits does so for workgroups that have started before
// it, and the first of those in line waits for nobody. (With one counter for all, its
// 13 ns for each workgroup were most of the time.) A pair and a state are one 64-bit word each, written and read by atomics
// of the device's scope: a word is either all there or still the mark that the
// clearing launch has left in it, and no order between words is relied on. Should a
// word never come (the workspace overwritten by somebody else's work), a wait gives
// up after kPolls looks and takes NaN.
//
// Bound by memory where the columns are many (8 x 2048 x 1536 channels, 192 columns: 52
// us for 201 MB, 3.9 of a large copy's 5.2 TB/s, with the vector ALU busy for half of it),
// and by the latency of looks and tickets where they are few (1 x 131072 x 256, 4 columns:
// 92 us for 268 MB, waves waiting for 60% of their time). Waves of 16 or 32 channels with
// more rows each, and workgroups that stay for another piece, were slower at both.
#include "glr_device.h"
#include "glr_launch.h"

namespace ssm {
namespace {

constexpr int kWaves = 4, kRows = 16, kPieceRows = kWaves * kRows;

constexpr int kFan = 16, kEach = kFan / kWaves;  // entries that a wave gathers at a time
constexpr int kPolls = 1 << 20;
constexpr uint64_t kMark = ~uint64_t{0};
constexpr int kCounterStep = 32;  // a cache line each

struct Chain {
  uint32_t* counters;  // one every kCounterStep, from -1 on
  uint64_t* pieces;  // (columns, pieces, 64), a column being 64 channels of a batch row
  uint64_t* groups;  // (columns, groups, 64)
  uint64_t* ranges;  // (columns, ranges, 64): the state entering range r + 1
  int n_pieces, n_groups, n_ranges, columns;
};

// All bits set: the mark, and -1.
__global__ __launch_bounds__(256) void glr_chain_clear(uint4* words, int64_t n) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += stride)
    words[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

// A word is never the mark: a NaN in its upper half goes out as the ordinary one.
__device__ __forceinline__ void publish(uint64_t* to, float P, float H) {
  const uint32_t h = H == H ? __float_as_uint(H) : 0x7fc00000u;
  __hip_atomic_store(to, static_cast<uint64_t>(h) << 32 | __float_as_uint(P), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t look(const uint64_t* from) {
  return __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The word at `from`, whose first look was `word`; every lane has its own.
__device__ __forceinline__ float2 await(const uint64_t* from, uint64_t word, int& polls) {
  while (__builtin_amdgcn_ballot_w64(word == kMark) != 0) {
    if (--polls < 0) return make_float2(1.0f, __builtin_nanf(""));
    __builtin_amdgcn_s_sleep(1);
    word = look(from);
  }
  return make_float2(__uint_as_float(static_cast<uint32_t>(word)), __uint_as_float(static_cast<uint32_t>(word >> 32)));
}
// First (P, H), then (p.x, p.y).
__device__ __forceinline__ void then(float& P, float& H, float2 p) {
  H = through(p.x, p.y, H);
  P = joined(P, p.x);
}

template <typename InT, int DECAY, int MIX, bool IN, bool Z, int W, int K>
__global__ __launch_bounds__(kLanes * W) void glr_chain(const GlrArgs g, const Chain chain) {
  __shared__ float2 pairs[W][kLanes];        // of the waves' rows
  __shared__ float2 gathered[2][W][kLanes];  // of the entries that the waves gather: pieces, groups
  __shared__ float entering[kLanes];         // the range
  __shared__ int ticket;
  const int lane = threadIdx.x % kLanes, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int column = blockIdx.x % chain.columns;
  if (threadIdx.x == 0)
    ticket = static_cast<int>(__hip_atomic_fetch_add(chain.counters + column * kCounterStep, 1u, __ATOMIC_RELAXED,
                                                     __HIP_MEMORY_SCOPE_AGENT) + 1);
  __syncthreads();
  const int piece = __builtin_amdgcn_readfirstlane(ticket);
  if (piece < 0 || piece >= chain.n_pieces) return;  // (a counter that somebody else has moved)
  const int batch = column / g.tiles, tile = column - batch * g.tiles;
  const int channel = tile * kLanes + lane, ch = min(channel, g.D - 1);
  const bool on = channel < g.D;
  const uint32_t at = static_cast<uint32_t>(ch) * sizeof(InT);
  const int64_t row0 = batch * g.L, state = static_cast<int64_t>(batch) * g.D + ch;
  const int L = static_cast<int>(g.L);
  const int t = piece * (W * K) + w * K, rows = max(0, min(K, L - t)), have = max(rows, 1);
  const int64_t row = row0 + min(t, L - 1);
  uint32_t u[K], dt[K], in[K], z[K];
  load_rows<InT, K>(g.dt, row, g.ds, have, at, dt);
  if (IN) load_rows<InT, K>(g.in, row, g.is, have, at, in);
  load_rows<InT, K>(g.u, row, g.us, have, at, u);
  if (Z) load_rows<InT, K>(g.z, row, g.zs, have, at, z);
  const uint32_t reset = reset_byte<K>(g.reset, row, rows, lane);
  const Channel<DECAY> c(g, ch);
  const float h0 = g.h0 && piece < kFan * kFan ? g.h0[state] : 0.0f;
  const uint32_t cuts = static_cast<uint32_t>(__builtin_amdgcn_ballot_w64(reset != 0));
  const bool plain = rows == K && cuts == 0;
  float a[K], b[K], P = 1.0f, H = 0.0f, none = 0.0f;
  bool cut = false;
  terms<InT, DECAY, MIX, IN, K>(c, u, dt, in, cuts, a, b);
  if (plain)
    run_rows<true, false, K>(a, b, b, K, 0, P, H, none, cut);
  else
    run_rows<false, false, K>(a, b, b, rows, cuts, P, H, none, cut);
  pairs[w][lane] = make_float2(cut ? kCut : P, H);
  __syncthreads();
  // what the waves before this one do to the piece's state, and (wave 0) what all of them do
  P = 1.0f;
  H = 0.0f;
  if (w == 0) {
#pragma unroll
    for (int i = 0; i < W; ++i) then(P, H, pairs[i][lane]);
    publish(chain.pieces + (static_cast<int64_t>(column) * chain.n_pieces + piece) * kLanes + lane, P, H);
    P = 1.0f;
    H = 0.0f;
  } else {
    for (int i = 0; i < w; ++i) then(P, H, pairs[i][lane]);
  }
  const float before_P = P, before_H = H;

  // First looks at all that this piece needs, then the waits.
  const int group = piece / kFan, range = group / kFan;
  const int first_piece = group * kFan + kEach * w, n_pieces = min(kEach, piece - first_piece);
  const int first_group = range * kFan + kEach * w, n_groups = min(kEach, group - first_group);
  const uint64_t* of_pieces =
      chain.pieces + (static_cast<int64_t>(column) * chain.n_pieces + first_piece) * kLanes + lane;
  const uint64_t* of_groups =
      chain.groups + (static_cast<int64_t>(column) * chain.n_groups + first_group) * kLanes + lane;
  const uint64_t* of_range =
      chain.ranges + (static_cast<int64_t>(column) * chain.n_ranges + range - 1) * kLanes + lane;
  const bool asks = range > 0 && w == W - 1;
  uint64_t pw[kEach], gw[kEach], rw = kMark;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    pw[i] = i < n_pieces ? look(of_pieces + i * kLanes) : kMark;
    gw[i] = i < n_groups ? look(of_groups + i * kLanes) : kMark;
  }
  if (asks) rw = look(of_range);
  int polls = kPolls;
  auto gather = [&](const uint64_t* from, int n, const uint64_t (&words)[kEach]) {
    P = 1.0f;
    H = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (i < n) then(P, H, await(from + i * kLanes, words[i], polls));
    return make_float2(P, H);
  };
  // What the group's pieces before this one do; known without waiting for any state.
  gathered[0][w][lane] = gather(of_pieces, n_pieces, pw);
  __syncthreads();
  float all_P = before_P, all_H = before_H;
  if (w == W - 1) {
    // the last wave knows what enters its own rows; its last row is the piece's last
    then(all_P, all_H, pairs[W - 1][lane]);
    if (piece % kFan == kFan - 1) {
      P = 1.0f;
      H = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) then(P, H, gathered[0][i][lane]);
      then(P, H, make_float2(all_P, all_H));
      publish(chain.groups + (static_cast<int64_t>(column) * chain.n_groups + group) * kLanes + lane, P, H);
    }
  }
  // The state that enters the range, and what its groups before this one do.
  float h = h0;
  if (group > 0) {
    gathered[1][w][lane] = gather(of_groups, n_groups, gw);
    if (asks) entering[lane] = await(of_range, rw, polls).y;
    __syncthreads();
    if (range > 0) h = entering[lane];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 p = gathered[1][i][lane];
      h = through(p.x, p.y, h);
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float2 p = gathered[0][i][lane];
    h = through(p.x, p.y, h);
  }
  if (w == W - 1) {
    const float after = through(all_P, all_H, h);
    if (piece % (kFan * kFan) == kFan * kFan - 1)
      publish(chain.ranges + (static_cast<int64_t>(column) * chain.n_ranges + range) * kLanes + lane, 1.0f, after);
    if (g.h_last && piece == chain.n_pieces - 1 && on) g.h_last[state] = after;
  }
  h = through(before_P, before_H, h);
  if (plain) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      h = __builtin_fmaf(a[k], h, b[k]);
      b[k] = Z ? h * silu_f32(widen<InT>(z[k])) : h;
    }
    if (on) store_rows<true, K>(g.out, row0 + t, g.D, K, ch, g.out_bf16, b);
  } else if (rows > 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      h = (cuts >> k) & 1 ? b[k] : __builtin_fmaf(a[k], h, b[k]);
      b[k] = Z ? h * silu_f32(widen<InT>(z[k])) : h;
    }
    if (on) store_rows<false, K>(g.out, row0 + t, g.D, rows, ch, g.out_bf16, b);
  }
}

struct RunChain {
  template <typename InT, int DECAY, int MIX, bool IN, bool Z>
  static hipError_t run(unsigned blocks, const GlrArgs& g, const Chain& chain, hipStream_t stream) {
    hipLaunchKernelGGL((glr_chain<InT, DECAY, MIX, IN, Z, kWaves, kRows>), dim3(blocks), dim3(kWaves * kLanes), 0,
                       stream, g, chain);
    return hipGetLastError();
  }
};

}  // namespace

GlrPieces plan_glr_chain(int64_t B, int64_t L, int64_t D) {
  GlrPieces p{};
  const int64_t columns = B * ((D + kLanes - 1) / kLanes);
  p.rows = kPieceRows;
  p.pieces = (L + kPieceRows - 1) / kPieceRows;
  p.waves = kWaves;
  const int64_t groups = (p.pieces + kFan - 1) / kFan, ranges = (groups + kFan - 1) / kFan;
  const size_t word = kLanes * sizeof(uint64_t) * static_cast<size_t>(columns);
  p.off_P = static_cast<size_t>(columns) * kCounterStep * sizeof(uint32_t);  // the counters come first
  p.off_H = p.off_P + word * p.pieces;
  p.off_starts = p.off_H + word * groups;
  p.bytes = p.off_starts + word * ranges;
  return p;
}

hipError_t launch_glr_chain(const GlrPlan& plan, const GlrPieces& p, void* workspace, hipStream_t stream) {
  const GlrArgs g = glr_args(plan);
  char* ws = static_cast<char*>(workspace);
  Chain c{};
  c.counters = reinterpret_cast<uint32_t*>(ws);
  c.pieces = reinterpret_cast<uint64_t*>(ws + p.off_P);
  c.groups = reinterpret_cast<uint64_t*>(ws + p.off_H);
  c.ranges = reinterpret_cast<uint64_t*>(ws + p.off_starts);
  c.n_pieces = static_cast<int>(p.pieces);
  c.n_groups = (c.n_pieces + kFan - 1) / kFan;
  c.n_ranges = (c.n_groups + kFan - 1) / kFan;
  c.columns = static_cast<int>(plan.B) * g.tiles;
  const int64_t words = static_cast<int64_t>(p.bytes / sizeof(uint4));
  const unsigned clear = static_cast<unsigned>(words + 255 < 256 * 2048 ? (words + 255) / 256 : 2048);
  SSM_LOG("launch glr_chain_clear: %lld words; grid %u x 256 threads", static_cast<long long>(words), clear);
  hipLaunchKernelGGL(glr_chain_clear, dim3(clear), dim3(256), 0, stream, reinterpret_cast<uint4*>(ws), words);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned blocks = static_cast<unsigned>(p.pieces * c.columns);
  SSM_LOG("launch glr_chain<%d waves of %d rows>: %d pieces; grid %u x %d threads", kWaves, kRows, c.n_pieces, blocks,
          kWaves * kLanes);
  return glr_pick<RunChain>(plan, blocks, g, c, stream);
}

}  // namespace ssm
