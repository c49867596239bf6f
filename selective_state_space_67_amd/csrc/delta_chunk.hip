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

#include "delta_chunk.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;

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
// take A_kj as it came out of K K^T. Two workgroups a CU: the second hides the serial
// parts (3072 chunks of 128 entries in 54 us; one workgroup 73, three 53, four, which
// spill, 104).
template <typename InT, int NP, int KS, bool VEC, bool BWD, bool ASYNC>
__global__ __launch_bounds__(kThreads, 2) void delta_chunk_prepare(const ChunkArgs a) {
  using Tile = TokenTile<NP, KS>;
  extern __shared__ __align__(16) uint16_t staged_tokens[];
  uint16_t* sk = staged_tokens;
  uint16_t* sq = staged_tokens + NP * Tile::kPart;
  __shared__ ChunkGates gates;
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
  if (w == 0)
    chunk_gates<InT>(a, b, h, chunk, reinterpret_cast<float*>(rec + (BWD ? kRecGatesBwd : kRecGates)), lane, &gates);

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

// ---- the walk over the chunks ----

// What a walk leaves: the outputs, a piece's effect on the state, or every chunk's
// first state and U (for the backward).
enum Walk { kOutputs, kAggregates, kStates };

struct ScanArgs {
  ChunkArgs c;
  int pieces, chunks_piece;
  int col_blocks;   // workgroups per (head, piece)
  int out_bf16, out_runs;  // out_runs: rows of out take whole 16-byte runs
  const float* h0;  // (bh, dk, dv) or null
  const float* starts;  // states of pieces 1 .. (bh, piece, 32 KS, cols), or null
  float* agg;       // aggregates walk: (bh, piece, 32 KS, 32 KS + cols)
  int cols;         // dv rounded up to 16
  void* out;
  float* h_last;
  float* states;    // states walk: (bh, chunk, 32 KS, cols)
  float* U;         // states walk: (bh, chunk, 64, cols)
  int64_t record_bytes, record_gates;
};

constexpr int kWaves = kThreads / 64;
constexpr int kBlockCols = 16 * kWaves;  // columns of the state per workgroup

// What a workgroup stages of one chunk, in bytes from the stage's start. T, the
// first OP parts of P and the scalars keep the record's order.
template <typename InT, int NP, int KS, Walk MODE, bool QLDS, int OP>
struct Stage {
  static constexpr int kK = 0;
  static constexpr int kQ = kK + TokenTile<NP, KS>::kBytes;
  static constexpr int kT = kQ + (MODE == kOutputs && QLDS ? TokenTile<NP, KS>::kBytes : 0);
  static constexpr int kP = kT + kTriBytes;
  static constexpr int kGates = kP + (MODE == kOutputs ? kTriBytes / 3 * OP : 0);
  static constexpr int kV = kGates + kGateFloats * 4;  // (64, kBlockCols) of InT
  static constexpr int kBytes = kV + kChunk * kBlockCols * static_cast<int>(sizeof(InT));
};

// Where the staging of a chunk reads.
template <typename InT>
struct ChunkSource {
  const InT* q;
  const InT* k;
  const InT* v;  // the chunk's first token, column 0 of the head
  const char* record;
  const char* gates;
  int n_tokens;
};

template <typename InT>
__device__ __forceinline__ ChunkSource<InT> chunk_source(const ScanArgs& w, int bh, int b, int h, int c) {
  const ChunkArgs& a = w.c;
  ChunkSource<InT> s;
  const int64_t t0 = static_cast<int64_t>(b) * a.L + static_cast<int64_t>(c) * kChunk;
  const int hk = h / a.group;
  s.q = static_cast<const InT*>(a.q) + t0 * a.qs + static_cast<int64_t>(hk) * a.dk;
  s.k = static_cast<const InT*>(a.k) + t0 * a.ks + static_cast<int64_t>(hk) * a.dk;
  s.v = static_cast<const InT*>(a.v) + t0 * a.vs + static_cast<int64_t>(h) * a.dv;
  s.record = a.records + (static_cast<int64_t>(bh) * a.chunks + c) * w.record_bytes;
  s.gates = s.record + w.record_gates;
  s.n_tokens = static_cast<int>(min(static_cast<int64_t>(kChunk), a.L - static_cast<int64_t>(c) * kChunk));
  return s;
}

// ASYNC staging: whole 16-byte runs straight into LDS, 1 KB a wave and instruction.
// Tokens past the end repeat the last one (their beta is 0, so they change
// nothing), columns past dv repeat the last ones (never stored). A lane's byte
// offsets from the chunk's first token are the same for every whole chunk.
struct LaneOffsets {
  uint32_t k, q, v[2];
};

__device__ __forceinline__ LaneOffsets lane_offsets(const ChunkArgs& a, int n_tokens, int col0, int lane, int wave) {
  LaneOffsets o;
  const int last = n_tokens - 1, row = min(wave * 16 + (lane & 15), last);  // wave w: row tile w
  o.k = static_cast<uint32_t>(row) * static_cast<uint32_t>(a.ks) * 2 + (lane >> 4) * 16;
  o.q = static_cast<uint32_t>(row) * static_cast<uint32_t>(a.qs) * 2 + (lane >> 4) * 16;
  const int col = max(0, min(col0 + (lane & 7) * 8, a.dv - 8));
#pragma unroll
  for (int i = 0; i < 2; ++i)  // 8 tokens of 64 columns
    o.v[i] = static_cast<uint32_t>(min((wave * 2 + i) * 8 + lane / 8, last)) * static_cast<uint32_t>(a.vs) * 2 + col * 2;
  return o;
}

template <typename InT, int KS, Walk MODE, int OP>
__device__ __forceinline__ void stage_async(char* st, const ChunkSource<InT>& s, const LaneOffsets& o, int lane,
                                            int wave) {
  using S = Stage<InT, 1, KS, MODE, true, OP>;
  static_assert(kWaves == 4, "row tile w and values 16 w .. of wave w");
  const char *k = reinterpret_cast<const char*>(s.k), *q = reinterpret_cast<const char*>(s.q);
  const char* v = reinterpret_cast<const char*>(s.v);
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    load_to_lds(k + i * 64 + o.k, st + S::kK + (wave * KS + i) * 1024);
    if constexpr (MODE == kOutputs) load_to_lds(q + i * 64 + o.q, st + S::kQ + (wave * KS + i) * 1024);
  }
  const uint32_t own = lane * 16;
  constexpr int kTri = (MODE == kOutputs ? kTriBytes + kTriBytes / 3 * OP : kTriBytes) / 1024;
#pragma unroll
  for (int i = 0; i < (kTri + kWaves - 1) / kWaves; ++i) {
    const int f = wave + i * kWaves;
    if (f < kTri) load_to_lds(s.record + f * 1024 + own, st + S::kT + f * 1024);
  }
  if (wave == 3) load_to_lds(s.gates + own, st + S::kGates);
#pragma unroll
  for (int i = 0; i < 2; ++i) load_to_lds(v + o.v[i], st + S::kV + (wave * 2 + i) * 1024);
}

// Staging through registers, for float32 and for rows that are not whole runs.
template <typename InT, int NP, int KS, bool VEC, Walk MODE, bool QLDS, int OP>
__device__ __forceinline__ void stage_sync(char* st, const ChunkArgs& a, const ChunkSource<InT>& s, int col0) {
  using S = Stage<InT, NP, KS, MODE, QLDS, OP>;
  stage_tokens<InT, NP, KS, VEC, kThreads>(reinterpret_cast<uint16_t*>(st + S::kK), s.k, a.ks, s.n_tokens, 0, a.dk);
  if constexpr (MODE == kOutputs && QLDS)
    stage_tokens<InT, NP, KS, VEC, kThreads>(reinterpret_cast<uint16_t*>(st + S::kQ), s.q, a.qs, s.n_tokens, 0, a.dk);
  constexpr int kRuns = (MODE == kOutputs ? kTriBytes + kTriBytes / 3 * OP : kTriBytes) / 16;
  for (int i = threadIdx.x; i < kRuns; i += kThreads)
    reinterpret_cast<u32x4*>(st + S::kT)[i] = reinterpret_cast<const u32x4*>(s.record)[i];
  reinterpret_cast<float*>(st + S::kGates)[threadIdx.x] = reinterpret_cast<const float*>(s.gates)[threadIdx.x];
  InT* v = reinterpret_cast<InT*>(st + S::kV);
#pragma unroll
  for (int i = 0; i < kChunk * kBlockCols / kThreads; ++i) {
    const int e = threadIdx.x + i * kThreads, token = e / kBlockCols, col = col0 + e % kBlockCols;
    InT x{};
    if (token < s.n_tokens && col >= 0 && col < a.dv) x = s.v[token * a.vs + col];
    v[e] = x;
  }
}

// One wave's walk over the chunks of a piece with 16 columns of the state.
// AGG: the aggregates walk (no read-out; the first 32 KS columns start from the
// identity). With two stages the next chunk is loaded while this one is worked on.
// OP: parts of the products that only the output sees; two (2^-17) where it is
// rounded to bfloat16 (2^-9).
template <typename InT, int NP, int KS, bool VEC, Walk MODE, bool QLDS, bool ASYNC, int STAGES, int OP>
__global__ __launch_bounds__(kThreads) void delta_chunk_scan(const ScanArgs s) {
  using Tile = TokenTile<NP, KS>;
  using S = Stage<InT, NP, KS, MODE, QLDS, OP>;
  constexpr int DKT = 2 * KS;  // row tiles of the state
  constexpr bool AGG = MODE == kAggregates, OUT = MODE == kOutputs;
  extern __shared__ __align__(16) char staged[];
  const ChunkArgs& a = s.c;
  const int lane = threadIdx.x % 64, wave = wave_index(), g4 = (lane >> 4) * 4;
  const int cb = blockIdx.x % s.col_blocks, rest = blockIdx.x / s.col_blocks;
  const int piece = rest % s.pieces, bh = rest / s.pieces;
  const int b = bh / a.Hv, h = bh - b * a.Hv;
  const int strip = cb * kWaves + wave;                            // 16-column strip
  const int col0 = (cb * kWaves - (AGG ? DKT : 0)) * 16;           // the workgroup's first column of v
  const int own = col0 + wave * 16 + (lane & 15);                  // the lane's
  const bool has_v = own >= 0 && own < a.dv;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

  f32x4 H[DKT];
#pragma unroll
  for (int m = 0; m < DKT; ++m) {
    H[m] = zero;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = state_row(m, g4, r);
      if (AGG) {
        if (strip * 16 + (lane & 15) == row) H[m][r] = 1.0f;
      } else if (piece > 0) {
        if (own < s.cols)
          H[m][r] = s.starts[((static_cast<int64_t>(bh) * s.pieces + piece) * (32 * KS) + row) * s.cols + own];
      } else if (s.h0 && row < a.dk && has_v) {
        H[m][r] = s.h0[(static_cast<int64_t>(bh) * a.dk + row) * a.dv + own];
      }
    }
  }

  const int c0 = piece * s.chunks_piece, c1 = min(a.chunks, c0 + s.chunks_piece);
  ChunkSource<InT> src = chunk_source<InT>(s, bh, b, h, c0);
  const LaneOffsets whole = lane_offsets(a, kChunk, col0, lane, wave);
  const auto stage = [&](char* st, const ChunkSource<InT>& from) {
    if constexpr (ASYNC)
      stage_async<InT, KS, MODE, OP>(
          st, from, from.n_tokens == kChunk ? whole : lane_offsets(a, from.n_tokens, col0, lane, wave), lane, wave);
    else
      stage_sync<InT, NP, KS, VEC, MODE, QLDS, OP>(st, a, from, col0);
  };
  if constexpr (STAGES == 2) stage(staged, src);
  for (int c = c0; c < c1; ++c) {
    char* st = staged + (STAGES == 2 ? ((c - c0) & 1) * S::kBytes : 0);
    ChunkSource<InT> next = src;
    next.q += kChunk * a.qs;
    next.k += kChunk * a.ks;
    next.v += kChunk * a.vs;
    next.record += s.record_bytes;
    next.gates += s.record_bytes;
    next.n_tokens = static_cast<int>(min(static_cast<int64_t>(kChunk), a.L - static_cast<int64_t>(c + 1) * kChunk));
    if constexpr (STAGES == 2) {
      wait_loads();
      __syncthreads();  // this stage is loaded, and the other one is no longer read
      if (c + 1 < c1) stage(staged + ((c + 1 - c0) & 1) * S::kBytes, next);
    } else {
      __syncthreads();  // the previous chunk is no longer read
      stage(st, src);
      wait_loads();
      __syncthreads();
    }
    const uint16_t* sk = reinterpret_cast<const uint16_t*>(st + S::kK);
    const uint16_t* sq = reinterpret_cast<const uint16_t*>(st + S::kQ);
    const float* gates = reinterpret_cast<const float*>(st + S::kGates);

    if constexpr (MODE == kStates) {  // in the waves' own layout: columns of the strips are 16 neighbours
      float* to = s.states + (static_cast<int64_t>(bh) * a.chunks + c) * (32 * KS) * s.cols + own;
#pragma unroll
      for (int m = 0; m < DKT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (own < s.cols) to[static_cast<int64_t>(state_row(m, g4, r)) * s.cols] = H[m][r];
    }
    f32x4 X[4] = {zero, zero, zero, zero}, Y[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Frag<3> hb = split8(H[2 * ks], H[2 * ks + 1]);
      Frag<NP> kf[4], qf[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        kf[m] = Tile::rows(sk, m, ks, lane);
        if constexpr (OUT) {
          if constexpr (QLDS)
            qf[m] = Tile::rows(sq, m, ks, lane);
          else
            qf[m] = rows_from_global<InT, VEC>(src.q, a.qs, src.n_tokens, a.dk, m, ks, lane);
        }
      }
      mma_n(kf, hb, X);
      if constexpr (OUT) mma_n<OP>(qf, hb, Y);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      f32x4 V = zero;
      if constexpr (sizeof(InT) == 2) {
        // the lane's column of tokens 16 m + g4 ..
        const u32x2 w = read_transposed(reinterpret_cast<const uint16_t*>(st + S::kV) +
                                        (m * 16 + g4 + ((lane & 15) >> 2)) * kBlockCols + wave * 16 + (lane & 3) * 4);
        V = f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                  __uint_as_float(w.y & 0xFFFF0000u)};
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          V[r] = reinterpret_cast<const float*>(st + S::kV)[(m * 16 + g4 + r) * kBlockCols + wave * 16 + (lane & 15)];
      }
      if (AGG && !has_v) V = zero;
      const f32x4 e0 = *reinterpret_cast<const f32x4*>(gates + kE0 + m * 16 + g4);
      const f32x4 be = *reinterpret_cast<const f32x4*>(gates + kBeta + m * 16 + g4);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        X[m][r] = be[r] * __builtin_fmaf(-e0[r], X[m][r], V[r]);
        Y[m][r] *= e0[r];
      }
    }
    f32x4 U[4] = {zero, zero, zero, zero};
    {
      const Frag<3> rb[2] = {split8(X[0], X[1]), split8(X[2], X[3])};
      mma_tri(reinterpret_cast<const uint16_t*>(st + S::kT), rb, lane, U);
    }
    if constexpr (OUT) {
      const Frag<3> ub[2] = {split8(U[0], U[1]), split8(U[2], U[3])};
      mma_tri<OP>(reinterpret_cast<const uint16_t*>(st + S::kP), ub, lane, Y);
    }
    if constexpr (MODE == kStates) {
      float* to = s.U + (static_cast<int64_t>(bh) * a.chunks + c) * kChunk * s.cols + own;
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (own < s.cols) to[(m * 16 + g4 + r) * s.cols] = U[m][r];
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) U[m] *= *reinterpret_cast<const f32x4*>(gates + kEC + m * 16 + g4);
    const Frag<3> ub[2] = {split8(U[0], U[1]), split8(U[2], U[3])};
    const float aC = gates[kAC];
#pragma unroll
    for (int m = 0; m < DKT; ++m) H[m] *= aC;
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      Frag<NP> kc[DKT];
#pragma unroll
      for (int m = 0; m < DKT; ++m) kc[m] = Tile::columns(sk, m, ts, lane);
      mma_n(kc, ub[ts], H);
    }

    if constexpr (OUT) {
      const int64_t row0 = (static_cast<int64_t>(b) * a.L + static_cast<int64_t>(c) * kChunk) * a.Hv + h;  // x dv
      if (OP == 2 && (ASYNC || s.out_runs)) {  // ASYNC has whole runs everywhere
        // The strip's place among the staged values is this wave's alone and has been
        // read: the outputs turn there from columns to rows, 16 bytes a lane.
        uint16_t* o = reinterpret_cast<uint16_t*>(st + S::kV) + wave * 16;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int r = 0; r < 4; r += 2) {
            const uint32_t w = bf16_words(a.scale * Y[m][r], a.scale * Y[m][r + 1]);
            uint16_t* p = o + (m * 16 + g4 + r) * kBlockCols + (lane & 15);
            p[0] = static_cast<uint16_t>(w);
            p[kBlockCols] = static_cast<uint16_t>(w >> 16);
          }
        char* dst = static_cast<char*>(s.out) + (row0 * a.dv + col0 + wave * 16) * 2;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int token = i * 32 + lane / 2, half = (lane & 1) * 8;
          const u32x4 w = *reinterpret_cast<const u32x4*>(o + token * kBlockCols + half);
          if (token < src.n_tokens && col0 + wave * 16 + half < a.dv)
            *reinterpret_cast<u32x4*>(dst + static_cast<uint32_t>(token * a.Hv * a.dv + half) * 2) = w;
        }
      } else {
        const int64_t step = static_cast<int64_t>(a.Hv) * a.dv;  // elements between tokens
        const int64_t lane0 = row0 * a.dv + g4 * step + own;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (!has_v || m * 16 + g4 + r >= src.n_tokens) continue;
            if (OP == 2 || s.out_bf16)
              store_elem(static_cast<bf16_t*>(s.out) + (m * 16 + r) * step, lane0, a.scale * Y[m][r]);
            else
              store_elem(static_cast<float*>(s.out) + (m * 16 + r) * step, lane0, a.scale * Y[m][r]);
          }
      }
    }
    src = next;
  }

  if (AGG) {
    const int width = 32 * KS + s.cols, at = strip * 16 + (lane & 15);
    if (at >= width) return;
    float* dst = s.agg + (static_cast<int64_t>(bh) * s.pieces + piece) * (32 * KS) * width + at;
#pragma unroll
    for (int m = 0; m < DKT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) dst[static_cast<int64_t>(state_row(m, g4, r)) * width] = H[m][r];
  } else if (OUT && s.h_last && c1 == a.chunks && has_v) {
#pragma unroll
    for (int m = 0; m < DKT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = state_row(m, g4, r);
        if (row < a.dk) s.h_last[(static_cast<int64_t>(bh) * a.dk + row) * a.dv + own] = H[m][r];
      }
  }
}

// The states that pieces 1 .. start from: S <- M S + N over the pieces, 16 columns
// and all rows a workgroup, its waves sharing the rows. The next piece's
// operands are loaded before the current ones are used.
struct FoldArgs {
  const float* agg;
  const float* h0;
  float* starts;
  int pieces, dk, dv, cols, strips;
};

template <int KS>
__global__ __launch_bounds__(2 * KS * 64) void delta_fold(const FoldArgs a) {
  constexpr int ROWS = 32 * KS;
  __shared__ u32x4 S[2][KS][3][64];  // the state as B operand, two pieces in turn
  const int lane = threadIdx.x % 64, w = wave_index(), g4 = (lane >> 4) * 4;  // wave w: row tile w
  const int bh = blockIdx.x / a.strips, own = (blockIdx.x - bh * a.strips) * 16 + (lane & 15);
  const int width = ROWS + a.cols;
  f32x4 H;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = state_row(w, g4, r);
    H[r] = a.h0 && row < a.dk && own < a.dv ? a.h0[(static_cast<int64_t>(bh) * a.dk + row) * a.dv + own] : 0.0f;
  }
  const float* M = a.agg + static_cast<int64_t>(bh) * a.pieces * ROWS * width;
  f32x4 m[KS][2], n;
  const auto fetch = [&](int piece) {
    const float* p = M + static_cast<int64_t>(piece) * ROWS * width;
    const float* row = p + static_cast<int64_t>(state_row(w, lane & 12, lane & 3)) * width + 2 * g4;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      m[ks][0] = *reinterpret_cast<const f32x4*>(row + 32 * ks);
      m[ks][1] = *reinterpret_cast<const f32x4*>(row + 32 * ks + 4);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) n[r] = p[static_cast<int64_t>(state_row(w, g4, r)) * width + ROWS + own];
  };
  fetch(0);
  for (int piece = 0; piece + 1 < a.pieces; ++piece) {
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
    if (piece + 2 < a.pieces) fetch(piece + 1);
    __syncthreads();  // one barrier a piece: the other buffer was last read before the previous one
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      Frag<3> sb;
#pragma unroll
      for (int i = 0; i < 3; ++i) sb.p[i] = S[buf][ks][i][lane];
      H = mma(mf[ks], sb, H);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      a.starts[((static_cast<int64_t>(bh) * a.pieces + piece + 1) * ROWS + state_row(w, g4, r)) * a.cols + own] = H[r];
  }
}

template <typename InT, int NP, int KS, bool VEC, Walk MODE, bool QLDS, bool ASYNC, int OP>
hipError_t launch_walk(const ScanArgs& s, int64_t blocks, hipStream_t stream) {
  constexpr int kBytes = Stage<InT, NP, KS, MODE, QLDS, OP>::kBytes;
  constexpr int STAGES = ASYNC && 2 * kBytes <= kMaxLds ? 2 : 1;
  static_assert(kBytes <= kMaxLds, "a chunk's stage exceeds LDS");
  SSM_LOG("launch delta_chunk_scan<%d parts, %d rows, walk %d>: %d pieces of %d chunks, %d stages of %d bytes; "
          "grid %lld x %d threads",
          NP, 32 * KS, MODE, s.pieces, s.chunks_piece, STAGES, kBytes, static_cast<long long>(blocks), kThreads);
  hipLaunchKernelGGL((delta_chunk_scan<InT, NP, KS, VEC, MODE, QLDS, ASYNC, STAGES, OP>),
                     dim3(static_cast<unsigned>(blocks)), dim3(kThreads), STAGES * kBytes, stream, s);
  return hipGetLastError();
}

template <typename InT, int NP, int KS, bool VEC, bool ASYNC>
hipError_t launch_scan_ks(const DeltaPlan& p, const DeltaChunks& plan, ScanArgs s, hipStream_t stream) {
  // K and Q of a chunk side by side fit in LDS except for float32 past 128 entries
  constexpr bool QLDS = Stage<InT, NP, KS, kOutputs, true, 3>::kBytes <= kMaxLds;
  const int64_t heads = p.B * p.Hv;
  if (plan.pieces > 1) {
    const int strips = 2 * KS + s.cols / 16;
    s.col_blocks = (strips + kWaves - 1) / kWaves;
    hipError_t e = launch_walk<InT, NP, KS, VEC, kAggregates, QLDS, ASYNC, 3>(s, heads * plan.pieces * s.col_blocks, stream);
    if (e != hipSuccess) return e;
    FoldArgs f{s.agg, s.h0, const_cast<float*>(s.starts), plan.pieces, p.dk, p.dv, s.cols, s.cols / 16};
    SSM_LOG("launch delta_fold<%d rows>: grid %lld x %d threads", 32 * KS, static_cast<long long>(heads * f.strips),
            2 * KS * 64);
    hipLaunchKernelGGL((delta_fold<KS>), dim3(static_cast<unsigned>(heads * f.strips)), dim3(2 * KS * 64), 0, stream, f);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  s.col_blocks = (s.cols / 16 + kWaves - 1) / kWaves;
  const int64_t blocks = heads * plan.pieces * s.col_blocks;
  if (s.states) return launch_walk<InT, NP, KS, VEC, kStates, QLDS, ASYNC, 3>(s, blocks, stream);
  if (NP == 1 && s.out_bf16) return launch_walk<InT, NP, KS, VEC, kOutputs, QLDS, ASYNC, NP == 1 ? 2 : 3>(s, blocks, stream);
  return launch_walk<InT, NP, KS, VEC, kOutputs, QLDS, ASYNC, 3>(s, blocks, stream);
}

template <typename InT, int NP, bool VEC, bool ASYNC>
hipError_t launch_scan_vec(const DeltaPlan& p, const DeltaChunks& plan, const ScanArgs& s, hipStream_t stream) {
  switch (padded_ks(p.dk)) {
    case 1: return launch_scan_ks<InT, NP, 1, VEC, ASYNC>(p, plan, s, stream);
    case 2: return launch_scan_ks<InT, NP, 2, VEC, ASYNC>(p, plan, s, stream);
    case 3: return launch_scan_ks<InT, NP, 3, VEC, ASYNC>(p, plan, s, stream);
    case 4: return launch_scan_ks<InT, NP, 4, VEC, ASYNC>(p, plan, s, stream);
    case 6: return launch_scan_ks<InT, NP, 6, VEC, ASYNC>(p, plan, s, stream);
    default: return launch_scan_ks<InT, NP, 8, VEC, ASYNC>(p, plan, s, stream);
  }
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

hipError_t launch_chunk_prepare(const DeltaPlan& p, const ChunkArgs& a, bool bwd, hipStream_t stream) {
  const int64_t blocks = p.B * p.Hv * a.chunks;
  const bool vec = delta_vec(p);
  if (!p.in_bf16) return vec ? prepare_f32<true>(a, blocks, bwd, stream) : prepare_f32<false>(a, blocks, bwd, stream);
  if (vec && p.dk == 32 * padded_ks(p.dk)) return prepare_bf16<true, true>(a, blocks, bwd, stream);
  return vec ? prepare_bf16<true, false>(a, blocks, bwd, stream) : prepare_bf16<false, false>(a, blocks, bwd, stream);
}

DeltaChunks plan_delta_chunks(int64_t B, int64_t L, int Hv, int dk, int dv, int requested) {
  DeltaChunks d{};
  d.chunks = static_cast<int>((L + kChunk - 1) / kChunk);
  d.pieces = 1;
  if (requested > 0) d.pieces = std::min(requested, d.chunks);
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
  d.bytes = off;
  return d;
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
  const bool vec = delta_vec(p);
  if (!p.in_bf16)
    return vec ? launch_scan_vec<float, 3, true, false>(p, plan, s, stream)
               : launch_scan_vec<float, 3, false, false>(p, plan, s, stream);
  // Straight loads to LDS: rows that fill the padded tile, values in whole runs.
  const bool async = vec && p.dk == 32 * padded_ks(p.dk) && p.dv % 8 == 0 && p.vs % 8 == 0 && delta_aligned(p.v, 16) &&
                     p.qs < reach && p.ks < reach && p.vs < reach && (s.out_runs || !p.out_bf16);
  if (async) return launch_scan_vec<bf16_t, 1, true, true>(p, plan, s, stream);
  return vec ? launch_scan_vec<bf16_t, 1, true, false>(p, plan, s, stream)
             : launch_scan_vec<bf16_t, 1, false, false>(p, plan, s, stream);
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
  if (plan.pieces > 1) {
    s.agg = reinterpret_cast<float*>(ws + plan.off_agg);
    s.starts = reinterpret_cast<float*>(ws + plan.off_starts);
  }
  s.out_bf16 = p.out_bf16;
  s.out = p.out;
  s.h_last = p.h_last;
  return launch_scan(p, plan, s, stream);
}

hipError_t launch_delta_states(const DeltaPlan& p, const ChunkArgs& c, float* states, float* U, hipStream_t stream) {
  DeltaChunks one{};
  one.chunks = one.chunks_piece = c.chunks;
  one.pieces = 1;
  ScanArgs s{};
  s.c = c;
  s.record_bytes = kRecBytesBwd;
  s.record_gates = kRecGatesBwd;
  s.states = states;
  s.U = U;
  return launch_scan(p, one, s, stream);
}

}  // namespace ssm
