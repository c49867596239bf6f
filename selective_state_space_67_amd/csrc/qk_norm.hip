// Norms of queries and keys for each head with the position rotation, and
// their gradients, in one pass over the data.
//
//   r = (sum x^2 + eps)^-1/2 or (mean x^2 + eps)^-1/2,  y = w (x r),  out = turn(y)
//   dz = turn^-1(dout),  dw = sum dz (x r),  dx = r (w dz - (x r) s (w dz . x r))
//
// Both directions are bound by memory: each element is read once and written
// once (the backward reads x and the output's gradient). A head's row is cut into
// slots of 2 V entries, one or two slots a lane, LR lanes a row. In the turned
// part a slot holds V entries of each side of the rotation, (i, i + rot/2) or
// neighbours, so no lane needs another's entries and the only exchange is the
// sum over the row's lanes. A group of lanes keeps its token while it goes
// through the heads, so the token's angles are loaded once.
//
// V = 4 (16 bytes of bfloat16 a slot) needs sizes and addresses in multiples of
// a slot; V = 1 takes everything else.
#include <algorithm>

#include "device_math.h"
#include "kernels_delta.h"
#include "lane_sums.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;

struct NormArgs {
  int64_t tokens, L, P;
  int64_t first;                      // lane group that the launch starts with (forward)
  int Hq, Hk, d, rot, slots, turned;  // turned: slots of the rotated part
  int parts, heads_part;              // a token's heads are split over `parts` lane groups
  const void* q;
  const void* k;
  int64_t qs, ks;
  const float* wq;
  const float* wk;
  const float* cos;
  const float* sin;
  const int32_t* positions;
  void* q_out;
  void* k_out;
  const void* dq_out;
  const void* dk_out;
  void* dq;
  void* dk;
  float* part;
  float eps, share;  // share: 1 (L2) or 1 / d (RMS)
  int interleaved;
};

// Where a slot's two runs of V entries lie, and its first pair's place in the
// table (V pairs a slot). A run at `none` does not exist.
struct Slot {
  int e0, e1, pair;  // pair < 0: not turned
  bool on, second;
};

template <int V>
__device__ __forceinline__ Slot slot_of(const NormArgs& a, int j) {
  Slot s;
  s.on = j < a.slots;
  s.second = s.on;
  s.pair = -1;
  if (j < a.turned) {
    s.pair = j * V;
    s.e0 = a.interleaved ? 2 * V * j : V * j;
    s.e1 = a.interleaved ? s.e0 + V : a.rot / 2 + V * j;
  } else {
    s.e0 = a.rot + 2 * V * (j - a.turned);
    s.e1 = s.e0 + V;
    if (s.e1 >= a.d) s.second = false;  // an odd rest (V = 1)
  }
  return s;
}

template <typename T, int V>
__device__ __forceinline__ void load_slot(const T* row, const Slot& s, float (&x)[2 * V]) {
#pragma unroll
  for (int i = 0; i < 2 * V; ++i) x[i] = 0.0f;
  if (!s.on) return;
  if constexpr (V == 1) {
    x[0] = load_elem(row, s.e0);
    if (s.second) x[1] = load_elem(row, s.e1);
  } else {
    const typename Run<T, V>::raw u = Run<T, V>::load(row + s.e0), v = Run<T, V>::load(row + s.e1);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = Run<T, V>::at(u, i);
      x[V + i] = Run<T, V>::at(v, i);
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_slot(T* row, const Slot& s, const float (&x)[2 * V]) {
  if (!s.on) return;
  if constexpr (V == 1) {
    store_elem(row, s.e0, x[0]);
    if (s.second) store_elem(row, s.e1, x[1]);
  } else {
    float lo[V], hi[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      lo[i] = x[i];
      hi[i] = x[V + i];
    }
    store_run<V>(row + s.e0, lo);
    store_run<V>(row + s.e1, hi);
  }
}

// The slot's pairs turned by their angles; back: by the opposite angles.
template <int V, bool BACK>
__device__ __forceinline__ void turn(const NormArgs& a, const Slot& s, const float (&c)[V], const float (&sn)[V],
                                     float (&x)[2 * V]) {
  if (s.pair < 0) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float co = c[i], si = BACK ? -sn[i] : sn[i];
    if (V > 1 && a.interleaved) {
      const float p = x[2 * i], q = x[2 * i + 1];
      x[2 * i] = __builtin_fmaf(p, co, -q * si);
      x[2 * i + 1] = __builtin_fmaf(q, co, p * si);
    } else {
      const float p = x[i], q = x[V + i];
      x[i] = __builtin_fmaf(p, co, -q * si);
      x[V + i] = __builtin_fmaf(q, co, p * si);
    }
  }
}

// A token's angles for a lane's slots; NaN where its position has none.
template <int V, int NS>
__device__ __forceinline__ void load_angles(const NormArgs& a, int64_t token, const Slot (&s)[NS], float (&c)[NS][V],
                                            float (&sn)[NS][V]) {
  if (a.rot == 0) return;
  const int64_t pos = a.positions ? a.positions[token] : token % a.L;
  const bool known = pos >= 0 && pos < a.P;
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    if (s[j].pair < 0 || !s[j].on) continue;
    const int64_t at = pos * (a.rot / 2) + s[j].pair;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[j][i] = known ? a.cos[at + i] : __builtin_nanf("");
      sn[j][i] = known ? a.sin[at + i] : __builtin_nanf("");
    }
  }
}

template <typename InT, int V, int LR, int NS>
__device__ __forceinline__ float row_factor(const NormArgs& a, const float (&x)[NS][2 * V]) {
  float sq = 0.0f;
#pragma unroll
  for (int j = 0; j < NS; ++j)
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) sq = __builtin_fmaf(x[j][i], x[j][i], sq);
  return __builtin_amdgcn_rsqf(__builtin_fmaf(lanes_sum<LR>(sq), a.share, a.eps));
}

template <int V, int NS>
__device__ __forceinline__ void load_weights(const float* w, const Slot (&s)[NS], float (&x)[NS][2 * V]) {
#pragma unroll
  for (int j = 0; j < NS; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[j][i] = w && s[j].on ? w[s[j].e0 + i] : 1.0f;
      x[j][V + i] = w && s[j].second ? w[s[j].e1 + i] : 1.0f;
    }
}

template <typename InT, typename OutT, int V, int LR, int NS>
__global__ __launch_bounds__(kThreads) void qk_norm_fwd(const NormArgs a) {
  const int64_t group = a.first + static_cast<int64_t>(blockIdx.x) * (kThreads / LR) + threadIdx.x / LR;
  const int64_t token = group / a.parts;
  if (token >= a.tokens) return;  // whole groups; the sums stay inside a group
  const int lane = threadIdx.x % LR;
  Slot s[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) s[j] = slot_of<V>(a, j * LR + lane);
  float c[NS][V], sn[NS][V], w[NS][2 * V];
  load_angles<V, NS>(a, token, s, c, sn);
  const int first = static_cast<int>(group - token * a.parts) * a.heads_part;
  const int last = min(first + a.heads_part, a.Hq + a.Hk);
  for (int head = first; head < last; ++head) {
    const bool is_q = head < a.Hq;
    const int hh = is_q ? head : head - a.Hq;
    if (head == first || head == a.Hq) load_weights<V, NS>(is_q ? a.wq : a.wk, s, w);
    const InT* row = static_cast<const InT*>(is_q ? a.q : a.k) + token * (is_q ? a.qs : a.ks) +
                     static_cast<int64_t>(hh) * a.d;
    OutT* dst = static_cast<OutT*>(is_q ? a.q_out : a.k_out) + (token * (is_q ? a.Hq : a.Hk) + hh) * a.d;
    float x[NS][2 * V];
#pragma unroll
    for (int j = 0; j < NS; ++j) load_slot<InT, V>(row, s[j], x[j]);
    const float r = row_factor<InT, V, LR, NS>(a, x);
#pragma unroll
    for (int j = 0; j < NS; ++j) {
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) x[j][i] = x[j][i] * r * w[j][i];
      turn<V, false>(a, s[j], c[j], sn[j], x[j]);
      store_slot<OutT, V>(dst, s[j], x[j]);
    }
  }
}

// A head of one entry has nothing across its own direction: w dz - (x r) s (w dz . x r)
// is then w dz (1 - s (x r)^2) = w dz eps r^2, taken in that form, since the
// difference would lose what is left of it.
//
// The workgroups go through the (token, part) items in strides; each lane keeps
// its slots' weight gradients in registers, a workgroup adds its groups' in a
// fixed order and writes one row of 2 d sums (q's, then k's).
template <typename InT, typename OutT, int V, int LR, int NS>
__global__ __launch_bounds__(kThreads) void qk_norm_bwd(const NormArgs a) {
  extern __shared__ float sums[];  // (groups, 2 d)
  constexpr int kGroups = kThreads / LR;
  const int lane = threadIdx.x % LR, mine = threadIdx.x / LR;
  Slot s[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) s[j] = slot_of<V>(a, j * LR + lane);
  float dwq[NS][2 * V] = {}, dwk[NS][2 * V] = {};
  const int64_t items = a.tokens * a.parts, stride = static_cast<int64_t>(gridDim.x) * kGroups;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kGroups + mine; item < items; item += stride) {
    const int64_t token = item / a.parts;
    float c[NS][V], sn[NS][V], w[NS][2 * V];
    load_angles<V, NS>(a, token, s, c, sn);
    const int first = static_cast<int>(item - token * a.parts) * a.heads_part;
    const int last = min(first + a.heads_part, a.Hq + a.Hk);
    for (int head = first; head < last; ++head) {
      const bool is_q = head < a.Hq;
      const int hh = is_q ? head : head - a.Hq;
      if (head == first || head == a.Hq) load_weights<V, NS>(is_q ? a.wq : a.wk, s, w);
      const InT* row = static_cast<const InT*>(is_q ? a.q : a.k) + token * (is_q ? a.qs : a.ks) +
                       static_cast<int64_t>(hh) * a.d;
      const int64_t at = (token * (is_q ? a.Hq : a.Hk) + hh) * a.d;
      const InT* grow = static_cast<const InT*>(is_q ? a.dq_out : a.dk_out) + at;
      float x[NS][2 * V], dz[NS][2 * V];
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        load_slot<InT, V>(row, s[j], x[j]);
        load_slot<InT, V>(grow, s[j], dz[j]);
      }
      const float r = row_factor<InT, V, LR, NS>(a, x);
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        turn<V, true>(a, s[j], c[j], sn[j], dz[j]);
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) {
          x[j][i] *= r;  // the normed row
          const float g = dz[j][i] * x[j][i];
          if (is_q)
            dwq[j][i] += g;
          else
            dwk[j][i] += g;
          dz[j][i] *= w[j][i];
          dot = __builtin_fmaf(dz[j][i], x[j][i], dot);
        }
      }
      dot = lanes_sum<LR>(dot) * a.share;
      OutT* dst = static_cast<OutT*>(is_q ? a.dq : a.dk) + at;
#pragma unroll
      for (int j = 0; j < NS; ++j) {
#pragma unroll
        for (int i = 0; i < 2 * V; ++i)
          dz[j][i] = r * (V == 1 && a.d == 1 ? dz[j][i] * (a.eps * r * r) : __builtin_fmaf(-x[j][i], dot, dz[j][i]));
        store_slot<OutT, V>(dst, s[j], dz[j]);
      }
    }
  }
  if (!a.part) return;
  float* row = sums + mine * 2 * a.d;
#pragma unroll
  for (int j = 0; j < NS; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (s[j].on) {
        row[s[j].e0 + i] = dwq[j][i];
        row[a.d + s[j].e0 + i] = dwk[j][i];
      }
      if (s[j].second) {
        row[s[j].e1 + i] = dwq[j][V + i];
        row[a.d + s[j].e1 + i] = dwk[j][V + i];
      }
    }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * a.d; e += kThreads) {
    float t = 0.0f;
    for (int g = 0; g < kGroups; ++g) t += sums[g * 2 * a.d + e];
    a.part[static_cast<int64_t>(blockIdx.x) * 2 * a.d + e] = t;
  }
}

// dwq and dwk from the workgroups' rows: 16 entries a workgroup, 16 threads an
// entry, each adding every 16th row in order, then the 16 sums in order. A thread has
// eight rows under way: one at a time, 1024 rows took 20 us, a fifth of the backward.
__global__ __launch_bounds__(kThreads) void qk_norm_reduce(const float* __restrict__ part, float* dwq, float* dwk,
                                                           int rows, int d) {
  constexpr int kAhead = 8;
  __shared__ float t[16][17];
  const int col = threadIdx.x % 16, by = threadIdx.x / 16, e = blockIdx.x * 16 + col;
  float x = 0.0f;
  if (e < 2 * d)
    for (int r = by; r < rows; r += 16 * kAhead) {
      float row[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        row[i] = r + 16 * i < rows ? part[static_cast<int64_t>(r + 16 * i) * 2 * d + e] : 0.0f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) x += row[i];
    }
  t[by][col] = x;
  __syncthreads();
  if (by != 0 || e >= 2 * d) return;
  x = 0.0f;
  for (int r = 0; r < 16; ++r) x += t[r][col];
  float* dst = e < d ? dwq : dwk;
  if (dst) dst[e < d ? e : e - d] = x;
}

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

NormArgs norm_args(const NormPlan& p) {
  NormArgs a{};
  a.tokens = p.B * p.L;
  a.L = p.L;
  a.P = p.P;
  a.Hq = p.Hq;
  a.Hk = p.Hk;
  a.d = p.d;
  a.rot = p.rot;
  a.q = p.q;
  a.k = p.k;
  a.qs = p.qs;
  a.ks = p.ks;
  a.wq = p.wq;
  a.wk = p.wk;
  a.cos = p.cos;
  a.sin = p.sin;
  a.positions = p.positions;
  a.q_out = p.q_out;
  a.k_out = p.k_out;
  a.dq_out = p.dq_out;
  a.dk_out = p.dk_out;
  a.dq = p.dq;
  a.dk = p.dk;
  a.eps = p.eps;
  a.share = p.l2 ? 1.0f : 1.0f / static_cast<float>(p.d);
  a.interleaved = p.interleaved;
  return a;
}

// Heads are split over lane groups until the launch has this many threads, 2048 of them a
// CU. The forward moves 8 x 2048 tokens of 2 x 12 heads of 128 in 47 us, 4.5 TB/s (a large
// copy reaches 5.2).
constexpr int64_t kWantThreads = int64_t{1} << 19;

template <typename InT, typename OutT, int V, int LR, int NS, bool BWD>
hipError_t launch(const NormPlan& p, NormArgs a, hipStream_t stream) {
  a.slots = a.rot / (2 * V) + (a.d - a.rot + 2 * V - 1) / (2 * V);
  a.turned = a.rot / (2 * V);
  const int heads = a.Hq + a.Hk;
  const int64_t want = (kWantThreads + a.tokens * LR - 1) / (a.tokens * LR);
  a.parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, heads)));
  a.heads_part = (heads + a.parts - 1) / a.parts;
  a.parts = (heads + a.heads_part - 1) / a.heads_part;
  constexpr int kGroups = kThreads / LR;
  const int64_t blocks = (a.tokens * a.parts + kGroups - 1) / kGroups;
  if constexpr (!BWD) {
    SSM_LOG("launch qk_norm_fwd<%d entries a run, %d lanes a row>: %d heads in %d parts; grid %lld x %d threads", V,
            LR, heads, a.parts, static_cast<long long>(blocks), kThreads);
    constexpr int64_t kMost = int64_t{1} << 23;  // workgroups a launch, which has less than 2^32 threads
    for (int64_t at = 0; at < blocks; at += kMost) {
      a.first = at * kGroups;
      hipLaunchKernelGGL((qk_norm_fwd<InT, OutT, V, LR, NS>), dim3(static_cast<unsigned>(std::min(kMost, blocks - at))),
                         dim3(kThreads), 0, stream, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  } else {
    const int rows = static_cast<int>(std::min<int64_t>(blocks, norm_bwd_blocks(a.tokens, heads, a.d)));
    a.part = p.dwq || p.dwk ? p.part : nullptr;
    const size_t lds = static_cast<size_t>(kGroups) * 2 * a.d * sizeof(float);
    SSM_LOG("launch qk_norm_bwd<%d entries a run, %d lanes a row>: %d heads in %d parts; grid %d x %d threads", V, LR,
            heads, a.parts, rows, kThreads);
    hipLaunchKernelGGL((qk_norm_bwd<InT, OutT, V, LR, NS>), dim3(rows), dim3(kThreads), lds, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part) return e;
    const int grid = (2 * a.d + 15) / 16;
    SSM_LOG("launch qk_norm_reduce: %d rows; grid %d x %d threads", rows, grid, kThreads);
    hipLaunchKernelGGL(qk_norm_reduce, dim3(grid), dim3(kThreads), 0, stream, a.part, p.dwq, p.dwk, rows, a.d);
    return hipGetLastError();
  }
}

template <typename InT, typename OutT, bool BWD>
hipError_t launch_types(const NormPlan& p, hipStream_t stream) {
  const NormArgs a = norm_args(p);
  const uintptr_t in4 = 4 * sizeof(InT), out4 = 4 * sizeof(OutT);
  bool runs = a.d % 8 == 0 && a.rot % 8 == 0 && aligned_to(a.q, in4) && aligned_to(a.k, in4) && a.qs % 4 == 0 &&
              a.ks % 4 == 0;
  if (BWD)
    runs = runs && aligned_to(a.dq_out, in4) && aligned_to(a.dk_out, in4) && aligned_to(a.dq, out4) &&
           aligned_to(a.dk, out4);
  else
    runs = runs && aligned_to(a.q_out, out4) && aligned_to(a.k_out, out4);
  if (runs) {
    if (a.d <= 32) return launch<InT, OutT, 4, 4, 1, BWD>(p, a, stream);
    if (a.d <= 64) return launch<InT, OutT, 4, 8, 1, BWD>(p, a, stream);
    if (a.d <= 128) return launch<InT, OutT, 4, 16, 1, BWD>(p, a, stream);
    return launch<InT, OutT, 4, 32, 1, BWD>(p, a, stream);
  }
  if (a.d <= 32) return launch<InT, OutT, 1, 16, 1, BWD>(p, a, stream);
  if (a.d <= 128) return launch<InT, OutT, 1, 64, 1, BWD>(p, a, stream);
  return launch<InT, OutT, 1, 64, 2, BWD>(p, a, stream);
}

template <bool BWD>
hipError_t launch_norm(const NormPlan& p, hipStream_t stream) {
  if (p.in_bf16)
    return p.out_bf16 ? launch_types<bf16_t, bf16_t, BWD>(p, stream) : launch_types<bf16_t, float, BWD>(p, stream);
  return p.out_bf16 ? launch_types<float, bf16_t, BWD>(p, stream) : launch_types<float, float, BWD>(p, stream);
}

}  // namespace

// Workgroups of the backward, each of which leaves a row of sums for the weights: one for
// every 32768 elements up to 1024 (8 x 2048 tokens of 2 x 12 heads of 128: 69 us, 4.4 TB/s, and 6
// for the rows' sums; with 2048 and 4096 workgroups 20 us more).
int norm_bwd_blocks(int64_t tokens, int heads, int d) {
  const int64_t want = (tokens * heads * d + 32767) / 32768;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, 1024)));
}

hipError_t launch_qk_norm(const NormPlan& p, hipStream_t stream) { return launch_norm<false>(p, stream); }

hipError_t launch_qk_norm_bwd(const NormPlan& p, hipStream_t stream) { return launch_norm<true>(p, stream); }

}  // namespace ssm
