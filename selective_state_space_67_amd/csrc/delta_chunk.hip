// Gated delta rule in chunks of 64 tokens, forward.
//
// Within a chunk that starts from the state H0, with G_i the sum of log decays
// through token i, M_ij = exp(G_i - G_j) for j <= i of the same document (else 0)
// and e0, eC, aC the decays from the start, to the end and across (delta_mfma.h):
//
//   A_ij = beta_i M_ij (k_i . k_j), j < i        T = (I + A)^-1
//   U    = T R,    R = beta (V - e0 (K H0))      (the rows u_t of the recurrence)
//   out  = scale (e0 (Q H0) + P U),   P = M o (Q K^T)
//   H1   = aC H0 + K^T (eC U)
//
// Two launches. delta_chunk_prepare computes T and P of all chunks in parallel
// (they do not depend on the state). delta_chunk_scan then walks the chunks in
// order; columns of the state are independent, so a wave owns 16 of them for one
// head and keeps the state, R and U in registers (delta_mfma.h: a product's result
// is the next one's operand as it lies). The waves of a workgroup share only the
// staged tokens of K and Q.
//
// A long sequence on few heads is split into pieces: a first walk finds each
// piece's effect on the state, which is affine, H -> M H + N (the columns of M
// are a walk from the identity without values); delta_fold carries the state
// across the pieces, and the full walk starts every piece from its own state.
#include <algorithm>
#include <cmath>

#include "delta_walk.h"

namespace ssm {
namespace {

__device__ __forceinline__ f32x4 mfma4(f32x4 a, f32x4 b, f32x4 c) {  // 16 x 16 x 16 in float32
#pragma unroll
  for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
  return c;
}

// T, P (or T^T, P^T) and the scalars of one chunk of one head. Four waves; wave w
// makes row tile w of the 4 x 4 tiles of 16 tokens (and column tile w for the
// transposes).
//
// The triangular inverse is exact substitution, block by block: each 16 x 16
// diagonal block by forward substitution in float32, then, down a row,
//   T_ij = -(sum_{k=j+1..i} T_ik A_kj) T_jj
// with float32 matrix instructions. All blocks are used in the layout in which
// they were produced: the transposed products T_ij^T = -T_jj^T sum A_kj^T T_ik^T
// take A_kj as it came out of K K^T. Bound by the latency of that chain of small
// dependent products (the vector pipe is busy 18% of a wave's cycles); two workgroups a
// CU, one of which hides the serial parts of the other: 8 x 2048 x 12 heads of 128 entries in
// 48 us, 2.4 TB/s of records written (in an earlier form 54 us; one workgroup 73, three
// 53, four, which spill, 104).
template <typename InT, int NP, int KS, bool VEC, bool BWD, bool ASYNC>
__global__ __launch_bounds__(kThreads, 2) void delta_chunk_prepare(const ChunkArgs a) {
  using Tile = TokenTile<NP, KS>;
  extern __shared__ __align__(16) uint16_t staged_tokens[];
  uint16_t* sk = staged_tokens;
  uint16_t* sq = staged_tokens + NP * Tile::kPart;
  __shared__ __align__(16) float gates[kGateFloatsBwd];
  __shared__ float diag[4][16][20];  // A_ii, then T_ii; rows of 16 padded to 20
  const int lane = threadIdx.x % 64, g4 = (lane >> 4) * 4, col = lane & 15;
  const int w = wave_index();
  const int64_t record = blockIdx.x;
  const int bh = static_cast<int>(record / a.chunks), chunk = static_cast<int>(record - static_cast<int64_t>(bh) * a.chunks);
  const int b = bh / a.Hv, h = bh - b * a.Hv, hk = h / a.group;
  const int64_t t0 = static_cast<int64_t>(b) * a.L + static_cast<int64_t>(chunk) * kChunk;
  const int n_tokens = static_cast<int>(min(static_cast<int64_t>(kChunk), a.L - static_cast<int64_t>(chunk) * kChunk));
  const InT* q = static_cast<const InT*>(a.q) + t0 * a.qs + static_cast<int64_t>(hk) * a.dk;
  const InT* k = static_cast<const InT*>(a.k) + t0 * a.ks + static_cast<int64_t>(hk) * a.dk;

  char* rec = a.records + record * (BWD ? kRecBytesBwd : kRecBytes);
  if constexpr (ASYNC) {  // on their way while the first wave works out the decays
    stage_tokens_async<KS>(sk, k, a.ks, n_tokens, lane, w);
    stage_tokens_async<KS>(sq, q, a.qs, n_tokens, lane, w);
  }
  if (w == 0) chunk_gates<InT>(a, b, h, chunk, gates, lane);

  // S[k][j]: rows k, columns j (j < k <= w, and the diagonal k = j = w); with BWD
  // also R[k][i]: rows k, columns i (w <= k < i). P[j]: rows j, columns w;
  // with BWD rows j >= w of Q, columns w of K.
  f32x4 S[4][4] = {}, R[4][4] = {}, P[4] = {};
  for (int d0 = 0; d0 < a.dk; d0 += 32 * KS) {
    if constexpr (ASYNC) {
      wait_loads();
    } else {
      if (d0 > 0) __syncthreads();
      stage_tokens<InT, NP, KS, VEC, kThreads>(sk, k, a.ks, n_tokens, d0, a.dk);
      stage_tokens<InT, NP, KS, VEC, kThreads>(sq, q, a.qs, n_tokens, d0, a.dk);
    }
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      Frag<NP> kf[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) kf[i] = Tile::rows(sk, i, ks, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < i; ++j) {
          if (i <= w) S[i][j] = mma(kf[i], kf[j], S[i][j]);
          if (BWD && j >= w) R[j][i] = mma(kf[j], kf[i], R[j][i]);
        }
        if (i == w) S[i][i] = mma(kf[i], kf[i], S[i][i]);
      }
      if constexpr (BWD) {
        const Frag<NP> kw = Tile::rows(sk, w, ks, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i >= w) P[i] = mma(Tile::rows(sq, i, ks, lane), kw, P[i]);
      } else {
        const Frag<NP> qw = Tile::rows(sq, w, ks, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j <= w) P[j] = mma(kf[j], qw, P[j]);
      }
    }
  }

  {  // the record's scalars
    float* to = reinterpret_cast<float*>(rec + (BWD ? kRecGatesBwd : kRecGates));
    to[threadIdx.x] = gates[threadIdx.x];
    if (BWD) to[kThreads + threadIdx.x] = gates[kThreads + threadIdx.x];
  }
  // Decays and betas.
  {
    RowDecay rows[4];
    ColDecay cols[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rows[i] = row_decay(gates, i * 16 + g4);
      cols[i] = col_decay(gates, i * 16 + col);
    }
    const ColDecay cw = col_decay(gates, w * 16 + col);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int j = 0; j < i; ++j) {
          if (i <= w) S[i][j][r] *= rows[i].beta[r] * decay_down(rows[i], r, cols[j]);
          if (BWD && j >= w) R[j][i][r] *= cols[i].beta * decay_up(rows[j], r, cols[i]);  // transposed: A_ij of the system
        }
        if (i == w) S[i][i][r] *= g4 + r > col ? rows[i].beta[r] * decay_down(rows[i], r, cw) : 0.0f;
        if (BWD && i >= w) P[i][r] *= i * 16 + g4 + r >= w * 16 + col ? decay_down(rows[i], r, cw) : 0.0f;
        if (!BWD && i <= w) P[i][r] *= i * 16 + g4 + r <= w * 16 + col ? decay_up(rows[i], r, cw) : 0.0f;
      }
    }
  }

  // The diagonal block: lane c of the first 16 makes column c of its inverse.
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i == w)
#pragma unroll
      for (int r = 0; r < 4; ++r) diag[w][g4 + r][col] = S[i][i][r];
  __syncthreads();
  float x[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    float v = r == col ? 1.0f : 0.0f;
#pragma unroll
    for (int m = 0; m < r; ++m) v = __builtin_fmaf(-diag[w][r][m], x[m], v);
    x[r] = v;
  }
  __syncthreads();
  if (lane < 16)
#pragma unroll
    for (int r = 0; r < 16; ++r) diag[w][r][col] = x[r];
  __syncthreads();

  // Row w, right to left: Tr[j] = T_wj^T (rows j, columns w).
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 Tr[4] = {zero, zero, zero, zero};
#pragma unroll
  for (int j = 3; j >= 0; --j) {
    if (j == w) Tr[j] = *reinterpret_cast<const f32x4*>(&diag[j][col][g4]);
    if (j >= w) continue;
    f32x4 sum = zero;
#pragma unroll
    for (int i = j + 1; i < 4; ++i)
      if (i <= w) sum = mfma4(S[i][j], Tr[i], sum);
    f32x4 t;
#pragma unroll
    for (int r = 0; r < 4; ++r) t[r] = -diag[j][g4 + r][col];
    Tr[j] = mfma4(t, sum, zero);
  }
  uint16_t* T = reinterpret_cast<uint16_t*>(rec + kRecT);
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
    if (ks <= w / 2) store_tri(T, tri_index(w, ks), lane, split8(Tr[2 * ks], Tr[2 * ks + 1]));
  if constexpr (!BWD) {
    uint16_t* Pm = reinterpret_cast<uint16_t*>(rec + kRecP);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks <= w / 2) store_tri(Pm, tri_index(w, ks), lane, split8(P[2 * ks], P[2 * ks + 1]));
  } else {
    // Column w, top to bottom: Tc[i] = T_iw (rows i, columns w).
    f32x4 Tc[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i == w)
#pragma unroll
        for (int r = 0; r < 4; ++r) Tc[i][r] = diag[i][g4 + r][col];
      if (i <= w) continue;
      f32x4 sum = zero;
#pragma unroll
      for (int m = 0; m < i; ++m)
        if (m >= w) sum = mfma4(R[m][i], Tc[m], sum);
      const f32x4 t = *reinterpret_cast<const f32x4*>(&diag[i][col][g4]);
      Tc[i] = mfma4(-t, sum, zero);
    }
    uint16_t* Tt = reinterpret_cast<uint16_t*>(rec + kRecTt);
    uint16_t* Pt = reinterpret_cast<uint16_t*>(rec + kRecPt);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks >= w / 2) {
        store_tri(Tt, tri_t_index(w, ks), lane, split8(Tc[2 * ks], Tc[2 * ks + 1]));
        store_tri(Pt, tri_t_index(w, ks), lane, split8(P[2 * ks], P[2 * ks + 1]));
      }
  }
}

template <typename InT, int NP, int KS, bool VEC, bool ASYNC>
hipError_t prepare_ks(const ChunkArgs& a, int64_t blocks, bool bwd, hipStream_t stream) {
  const size_t lds = 2 * TokenTile<NP, KS>::kBytes;
  SSM_LOG("launch delta_chunk_prepare<%d parts, %d entries a pass>: backward %d; grid %lld x %d threads", NP, 32 * KS,
          bwd, static_cast<long long>(blocks), kThreads);
  if (bwd)
    hipLaunchKernelGGL((delta_chunk_prepare<InT, NP, KS, VEC, true, ASYNC>), dim3(static_cast<unsigned>(blocks)),
                       dim3(kThreads), lds, stream, a);
  else
    hipLaunchKernelGGL((delta_chunk_prepare<InT, NP, KS, VEC, false, ASYNC>), dim3(static_cast<unsigned>(blocks)),
                       dim3(kThreads), lds, stream, a);
  return hipGetLastError();
}

// bfloat16 rows in one pass; float32, three times as large, 64 entries a pass.
template <bool VEC, bool ASYNC>
hipError_t prepare_bf16(const ChunkArgs& a, int64_t blocks, bool bwd, hipStream_t stream) {
  switch (padded_ks(a.dk)) {
    case 1: return prepare_ks<bf16_t, 1, 1, VEC, ASYNC>(a, blocks, bwd, stream);
    case 2: return prepare_ks<bf16_t, 1, 2, VEC, ASYNC>(a, blocks, bwd, stream);
    case 3: return prepare_ks<bf16_t, 1, 3, VEC, ASYNC>(a, blocks, bwd, stream);
    case 4: return prepare_ks<bf16_t, 1, 4, VEC, ASYNC>(a, blocks, bwd, stream);
    case 6: return prepare_ks<bf16_t, 1, 6, VEC, ASYNC>(a, blocks, bwd, stream);
    default: return prepare_ks<bf16_t, 1, 8, VEC, ASYNC>(a, blocks, bwd, stream);
  }
}

template <bool VEC>
hipError_t prepare_f32(const ChunkArgs& a, int64_t blocks, bool bwd, hipStream_t stream) {
  if (a.dk <= 32) return prepare_ks<float, 3, 1, VEC, false>(a, blocks, bwd, stream);
  return prepare_ks<float, 3, 2, VEC, false>(a, blocks, bwd, stream);
}

// The states that pieces 1 .. start from: S <- M S + N over the pieces, 16 columns
// and all rows a workgroup, its waves sharing the rows. The next piece's
// operands are loaded before the current ones are used. A chain over the pieces, bound by
// reading M: 2.4 us a piece of 128 x 128 (64 pieces on 2 heads 152 us). Loads two pieces
// ahead changed nothing.
//
// Many pieces are therefore folded in groups: COMPOSE makes each group's (M, N) from its
// pieces', from the identity for M and zero for N; the fold over the groups gives the
// states that they start from; and a fold inside every group the pieces'. (64 pieces on 2
// heads in 8 groups: 19 + 17 + 19 us; the call 591 -> 490.)
struct FoldArgs {
  const float* agg;     // (bh, pieces, ROWS, ROWS + cols)
  const float* turned;  // BACK: M^T (bh, pieces, ROWS, ROWS)
  const float* h0;      // of group 0, (bh, dk, dv) or null
  const float* from;    // of groups 1 .., (bh, groups, ROWS, cols)
  float* out;           // (bh, pieces, ROWS, cols); COMPOSE: (bh, groups, ROWS, ROWS + cols)
  int pieces, groups, group_pieces;
  int dk, dv, cols, strips;
};

// BACK: of the adjoint, from the last piece to the first (piece numbers count from the end):
// dH at a piece's start = M^T (dH at its end) + N, N from the reverse walk. M^T is written
// by the aggregates' walk (gathered from M instead, 16 heads of 192 x 128 took 84 us, so 29).
template <int KS, bool COMPOSE, bool BACK>
__global__ __launch_bounds__(2 * KS * 64) void delta_fold(const FoldArgs a) {
  constexpr int ROWS = 32 * KS;
  __shared__ u32x4 S[2][KS][3][64];  // the state as B operand, two pieces in turn
  const int lane = threadIdx.x % 64, w = wave_index(), g4 = (lane >> 4) * 4;  // wave w: row tile w
  const int strip = blockIdx.x % a.strips, chain = blockIdx.x / a.strips;
  const int group = chain % a.groups, bh = chain / a.groups;
  const int first = group * a.group_pieces, last = min(first + a.group_pieces, a.pieces);
  const int width = ROWS + a.cols;
  const int at = strip * 16 + (lane & 15) + (COMPOSE ? 0 : ROWS), own = at - ROWS;  // own < 0: a column of M
  f32x4 H;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = state_row(w, g4, r);
    if (COMPOSE)
      H[r] = row == at ? 1.0f : 0.0f;
    else if (group > 0)
      H[r] = a.from[((static_cast<int64_t>(bh) * a.groups + group) * ROWS + row) * a.cols + own];
    else
      H[r] = a.h0 && row < a.dk && own < a.dv ? a.h0[(static_cast<int64_t>(bh) * a.dk + row) * a.dv + own] : 0.0f;
  }
  const float* M = a.agg + static_cast<int64_t>(bh) * a.pieces * ROWS * width;
  f32x4 m[KS][2], n;
  const auto fetch = [&](int piece) {
    const float* p = M + static_cast<int64_t>(BACK ? a.pieces - 1 - piece : piece) * ROWS * width;
    const int own_row = state_row(w, lane & 12, lane & 3);
    const float* row =
        (BACK ? a.turned + ((static_cast<int64_t>(bh) * a.pieces + a.pieces - 1 - piece) * ROWS + own_row) * ROWS
              : p + static_cast<int64_t>(own_row) * width) + 2 * g4;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      m[ks][0] = *reinterpret_cast<const f32x4*>(row + 32 * ks);
      m[ks][1] = *reinterpret_cast<const f32x4*>(row + 32 * ks + 4);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) n[r] = own >= 0 ? p[static_cast<int64_t>(state_row(w, g4, r)) * width + at] : 0.0f;
  };
  const auto store = [&](int counted) {
    const int piece = BACK ? a.pieces - 1 - counted : counted;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      a.out[((static_cast<int64_t>(bh) * a.pieces + piece) * ROWS + state_row(w, g4, r)) * a.cols + own] = H[r];
  };
  if (!COMPOSE && group > 0) store(first);
  const int end = COMPOSE ? last : last - 1;  // the last piece's own effect is the full walk's
  if (first < end) fetch(first);
  for (int piece = first; piece < end; ++piece) {
    // half of operand w / 2: the wave's rows are its slots 4 (w % 2) ..
    uint32_t lo[3], hi[3];
    split_pair(H.x, H.y, lo);
    split_pair(H.z, H.w, hi);
    const int buf = piece & 1;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      reinterpret_cast<u32x2*>(&S[buf][w / 2][i][lane])[w % 2] = u32x2{lo[i], hi[i]};
    Frag<3> mf[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) mf[ks] = split8(m[ks][0], m[ks][1]);
    H = n;
    if (piece + 1 < end) fetch(piece + 1);
    __syncthreads();  // one barrier a piece: the other buffer was last read before the previous one
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      Frag<3> sb;
#pragma unroll
      for (int i = 0; i < 3; ++i) sb.p[i] = S[buf][ks][i][lane];
      H = mma(mf[ks], sb, H);
    }
    if (!COMPOSE) store(piece + 1);
  }
  if (COMPOSE) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      a.out[((static_cast<int64_t>(bh) * a.groups + group) * ROWS + state_row(w, g4, r)) * width + at] = H[r];
  }
}

template <int KS, bool COMPOSE, bool BACK>
hipError_t launch_fold(FoldArgs f, int64_t heads, hipStream_t stream) {
  f.strips = f.cols / 16 + (COMPOSE ? 2 * KS : 0);
  const int64_t blocks = heads * f.groups * f.strips;
  SSM_LOG("launch delta_fold<%d rows, compose %d, back %d>: %d pieces in %d groups; grid %lld x %d threads", 32 * KS,
          COMPOSE, BACK, f.pieces, f.groups, static_cast<long long>(blocks), 2 * KS * 64);
  hipLaunchKernelGGL((delta_fold<KS, COMPOSE, BACK>), dim3(static_cast<unsigned>(blocks)), dim3(2 * KS * 64), 0, stream, f);
  return hipGetLastError();
}

template <int KS, bool BACK>
hipError_t fold_ks(const FoldArgs& all, float* group_agg, float* group_starts, int64_t heads, hipStream_t stream) {
  if (all.groups > 1) {
    FoldArgs f = all;
    f.out = group_agg;
    hipError_t e = launch_fold<KS, true, BACK>(f, heads, stream);
    if (e != hipSuccess) return e;
    f = all;
    f.agg = group_agg;
    f.out = group_starts;
    f.pieces = f.group_pieces = all.groups;
    f.groups = 1;
    if ((e = launch_fold<KS, false, false>(f, heads, stream)) != hipSuccess) return e;
  }
  return launch_fold<KS, false, BACK>(all, heads, stream);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

template <bool BACK>
hipError_t fold_any(const DeltaPlan& p, const DeltaChunks& plan, const ScanArgs& s, const float* first,
                    hipStream_t stream) {
  FoldArgs f{};
  f.agg = s.agg;
  f.turned = s.turned;
  f.h0 = first;
  f.from = s.group_starts;
  f.out = const_cast<float*>(s.starts);
  f.pieces = plan.pieces;
  f.groups = plan.groups;
  f.group_pieces = plan.group_pieces;
  f.dk = p.dk;
  f.dv = p.dv;
  f.cols = (p.dv + 15) / 16 * 16;
  const int64_t heads = p.B * p.Hv;
  switch (padded_ks(p.dk)) {
    case 1: return fold_ks<1, BACK>(f, s.group_agg, s.group_starts, heads, stream);
    case 2: return fold_ks<2, BACK>(f, s.group_agg, s.group_starts, heads, stream);
    case 3: return fold_ks<3, BACK>(f, s.group_agg, s.group_starts, heads, stream);
    case 4: return fold_ks<4, BACK>(f, s.group_agg, s.group_starts, heads, stream);
    case 6: return fold_ks<6, BACK>(f, s.group_agg, s.group_starts, heads, stream);
    default: return fold_ks<8, BACK>(f, s.group_agg, s.group_starts, heads, stream);
  }
}

void piece_args(const DeltaChunks& plan, char* ws, ScanArgs& s) {
  if (plan.pieces <= 1) return;
  s.agg = reinterpret_cast<float*>(ws + plan.off_agg);
  s.starts = reinterpret_cast<float*>(ws + plan.off_starts);
  s.group_agg = reinterpret_cast<float*>(ws + plan.off_group_agg);
  s.group_starts = reinterpret_cast<float*>(ws + plan.off_group_starts);
  if (plan.off_turned) s.turned = reinterpret_cast<float*>(ws + plan.off_turned);
}

}  // namespace

hipError_t launch_delta_fold(const DeltaPlan& p, const DeltaChunks& plan, const ScanArgs& s, hipStream_t stream) {
  return fold_any<false>(p, plan, s, s.h0, stream);
}

hipError_t launch_delta_fold_back(const DeltaPlan& p, const DeltaChunks& plan, char* ws, const float* dh_last,
                                  hipStream_t stream) {
  ScanArgs s{};
  piece_args(plan, ws, s);
  return fold_any<true>(p, plan, s, dh_last, stream);
}

hipError_t launch_chunk_prepare(const DeltaPlan& p, const ChunkArgs& a, bool bwd, hipStream_t stream) {
  const int64_t blocks = p.B * p.Hv * a.chunks;
  const bool vec = delta_vec(p);
  if (!p.in_bf16) return vec ? prepare_f32<true>(a, blocks, bwd, stream) : prepare_f32<false>(a, blocks, bwd, stream);
  if (vec && p.dk == 32 * padded_ks(p.dk)) return prepare_bf16<true, true>(a, blocks, bwd, stream);
  return vec ? prepare_bf16<true, false>(a, blocks, bwd, stream) : prepare_bf16<false, false>(a, blocks, bwd, stream);
}

namespace {

// Up to this many pieces are folded one after another, more in groups.
constexpr int kFoldAlone = 16;

// Pieces that cost least, in units of a chunk's step of the full walk (about 5 us at 128 x
// 128): rounds of one workgroup a CU times the chunks of a piece, where a step of the
// aggregates' walk, which has a workgroup for every 64 of dk + dv columns, takes 0.7;
// a piece's fold takes 0.7 (of three folds over the root of the pieces, where there are
// groups); and two more launches. Measured at 128 x 128: 2 heads of 131072
// steps 10212 us in one piece, 502 in 64; 16 heads x 2 of 4096 336 us, 232 in 4; 12 x 8 of
// 2048 220 us (410 in two: the grid is full as it is). The costs are those of bfloat16 forward;
// the choice was compared with one piece for 172 sizes (both types; 32 x 32, 64 x 64, 128 x
// 128, 192 x 128, 256 x 64 and 256 x 256; 2 to 64 heads of 256 to 8192 steps), and for the
// backward, which uses it too: it splits 70 of them, 3.0 times as fast in the mean (up to 15; the
// backward 2.5, up to 11), and the worst loses 5% (bfloat16 256 x 64, 24 heads of 2048 steps,
// 280 us against 267; backward 812 against 763).
int choose_pieces(int64_t heads, int chunks, int dk, int dv) {
  constexpr int64_t kCUs = 256;
  const int64_t strips = (dv + 15) / 16, state_strips = 2 * padded_ks(dk);
  const int64_t walk = heads * ((strips + 3) / 4), agg = heads * ((strips + state_strips + 3) / 4);
  int best = 1;
  double least = static_cast<double>(chunks) * static_cast<double>((walk + kCUs - 1) / kCUs);
  for (int n = 2; n <= std::min(chunks / 2, 256); ++n) {
    const int steps = (chunks + n - 1) / n;
    const double fold = 0.7 * (n > kFoldAlone ? 3.0 * std::sqrt(static_cast<double>(n)) : n) + (n > kFoldAlone ? 2.0 : 0.0);
    const double cost = steps * (static_cast<double>((walk * n + kCUs - 1) / kCUs) +
                                 0.7 * static_cast<double>((agg * n + kCUs - 1) / kCUs)) + fold + 3.0;
    if (cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

}  // namespace

DeltaChunks plan_delta_chunks(int64_t B, int64_t L, int Hv, int dk, int dv, int requested) {
  DeltaChunks d{};
  d.chunks = static_cast<int>((L + kChunk - 1) / kChunk);
  d.pieces = requested > 0 ? std::min(requested, d.chunks) : choose_pieces(B * Hv, d.chunks, dk, dv);
  d.chunks_piece = (d.chunks + d.pieces - 1) / d.pieces;
  d.pieces = (d.chunks + d.chunks_piece - 1) / d.chunks_piece;
  const size_t records = static_cast<size_t>(B) * Hv * d.chunks;
  const size_t rows = 32 * static_cast<size_t>(padded_ks(dk)), cols = (static_cast<size_t>(dv) + 15) / 16 * 16;
  const size_t piece_heads = static_cast<size_t>(B) * Hv * d.pieces;
  size_t off = 0;
  d.off_records = off;
  off += records * kRecBytes;
  d.off_agg = off;
  if (d.pieces > 1) off += align256(piece_heads * rows * (rows + cols) * sizeof(float));
  d.off_starts = off;
  if (d.pieces > 1) off += align256(piece_heads * rows * cols * sizeof(float));
  // groups of about the root of the pieces, from where three folds are shorter than one
  d.groups = 1;
  d.group_pieces = d.pieces;
  if (d.pieces > kFoldAlone) {
    d.group_pieces = 1;
    while (d.group_pieces * d.group_pieces < d.pieces) ++d.group_pieces;
    d.groups = (d.pieces + d.group_pieces - 1) / d.group_pieces;
  }
  const size_t group_heads = static_cast<size_t>(B) * Hv * d.groups;
  d.off_group_agg = off;
  if (d.groups > 1) off += align256(group_heads * rows * (rows + cols) * sizeof(float));
  d.off_group_starts = off;
  if (d.groups > 1) off += align256(group_heads * rows * cols * sizeof(float));
  d.bytes = off;
  return d;
}

bool delta_grids_fit(int64_t heads, int dk, int dv, const DeltaChunks& d) {
  const int64_t strips = (dv + 15) / 16, state_strips = 2 * padded_ks(dk);
  bool fit = fits_launch(heads * d.chunks, kThreads) &&
             fits_launch(placed_blocks(heads * d.pieces, (strips + kWaves - 1) / kWaves), kThreads);
  if (d.pieces > 1)
    fit = fit && fits_launch(placed_blocks(heads * d.pieces, (strips + state_strips + kWaves - 1) / kWaves), kThreads) &&
          fits_launch(heads * d.groups * (strips + state_strips), 64 * state_strips);
  return fit;
}

namespace {

hipError_t launch_scan(const DeltaPlan& p, const DeltaChunks& plan, ScanArgs& s, hipStream_t stream) {
  s.pieces = plan.pieces;
  s.chunks_piece = plan.chunks_piece;
  s.h0 = p.h0;
  s.cols = (p.dv + 15) / 16 * 16;
  // a chunk's rows lie within 2^31 bytes (for 32-bit offsets)
  const int64_t reach = int64_t{1} << 24;  // elements a token
  s.out_runs = p.dv % 8 == 0 && delta_aligned(p.out, 16) && static_cast<int64_t>(p.Hv) * p.dv < reach;
  if (!p.in_bf16) return launch_walk_f32(p, plan, s, stream);
  // Straight loads to LDS: rows that fill the padded tile, values in whole runs.
  const bool direct = s.c.vec && p.dk == 32 * padded_ks(p.dk) && p.dv % 8 == 0 && p.vs % 8 == 0 && delta_aligned(p.v, 16) &&
                     p.qs < reach && p.ks < reach && p.vs < reach && (s.out_runs || !p.out_bf16);
  return direct ? launch_walk_bf16_direct(p, plan, s, stream) : launch_walk_bf16(p, plan, s, stream);
}

}  // namespace

hipError_t launch_delta_chunks(const DeltaPlan& p, const DeltaChunks& plan, void* workspace, hipStream_t stream) {
  char* ws = static_cast<char*>(workspace);
  ScanArgs s{};
  s.c = chunk_args(p, plan.chunks);
  s.c.records = ws + plan.off_records;
  s.record_bytes = kRecBytes;
  s.record_gates = kRecGates;
  const hipError_t e = launch_chunk_prepare(p, s.c, false, stream);
  if (e != hipSuccess) return e;
  piece_args(plan, ws, s);
  s.out_bf16 = p.out_bf16;
  s.out = p.out;
  s.h_last = p.h_last;
  return launch_scan(p, plan, s, stream);
}

hipError_t launch_delta_states(const DeltaPlan& p, const ChunkArgs& c, const DeltaChunks& plan, char* ws, float* states,
                               float* U, hipStream_t stream) {
  ScanArgs s{};
  s.c = c;
  s.record_bytes = kRecBytesBwd;
  s.record_gates = kRecGatesBwd;
  piece_args(plan, ws, s);
  s.states = states;
  s.U = U;
  return launch_scan(p, plan, s, stream);
}

}  // namespace ssm
