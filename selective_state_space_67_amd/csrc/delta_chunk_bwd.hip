// Gated delta rule in chunks of 64 tokens, backward.
//
// With the forward's chunk quantities (delta_chunk.hip), dO the gradient of the
// output times scale, dH1 the adjoint of the state after the chunk:
//
//   dU = P^T dO + eC (K dH1)            dR = T^T dU          dV = beta dR
//   dH0 = aC dH1 + Q^T (e0 dO) - K^T (beta e0 dR)
//   dP = M o (dO U^T) (j <= i),  dS = -beta M o (dR U^T) (j < i)
//   dQ = e0 (dO H0^T) + dP K
//   dK = [eC (U dH1^T) + dP^T Q + dS^T K] + [dS K - beta e0 (dR H0^T)]
//   d beta_raw_i = (dR_i . U_i) (1 - beta_i / beta_scale)
//   d g_t = sum over i >= t of q_i . dQ_i + k_i . (second bracket - first without eC)_i
//         + sum over j < t of k_j . (eC (U dH1^T))_j + aC <dH1, H0>
//
// (M carries exp(G_i - G_j): the first bracket holds k as the j side of every decay,
// the second as its i side, and what has its sides before and from step t on crosses
// its decay. Pairs i = j cross nothing: their products are left out of the sum and
// added to dQ and dK afterwards, so that they need not cancel.)
//
// Five launches and a sum: the chunks' matrices (delta_chunk.hip, with transposes); the
// forward walk again, keeping each chunk's first state and U; the reverse walk
// below, which mirrors the forward one (a wave owns 16 columns of dH in registers)
// and keeps each chunk's dH1 and dR; the gradients of q and k, every chunk of every
// key head in parallel, with the value heads of a key head added up in one workgroup;
// and those of the gates, a wave for every chunk of every value head.
#include <algorithm>

#include "delta_chunk.h"
#include "lane_sums.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kBlockCols = 16 * kWaves;

struct BwdArgs {
  ChunkArgs c;
  int col_blocks, cols;
  int heads;             // batch rows x value heads
  int pieces, chunks_piece;  // of the reverse walk
  const float* ends;     // dH at the ends of pieces 0 .. pieces - 2 (bh, piece, 32 KS, cols)
  float* agg;            // not null: from dH = 0 at every piece's end, only what its start has, to
                         // the last cols columns of (bh, piece, 32 KS, 32 KS + cols)
  int items;             // chunks of all key heads
  int grad_bf16;
  bool vec_out;          // rows of dout come as whole 16-byte runs
  const void* dout;
  const float* dh_last;
  const float* states;   // (bh, chunk, 32 KS, cols)
  const float* U;        // (bh, chunk, 64, cols)
  float* dstates;        // as states: dH1
  float* dR;             // as U
  float* sums;           // (bh, chunk, split, kSumFloats): what the gates' gradients are made of
  float* part;           // (bh, chunk, 2): dA, d dt_bias
  void* dq;
  void* dk;
  void* dv;
  void* ddt;
  void* dbr;
  float* dh0;
};

template <typename InT, int NP, int KS, bool BOTH>
struct RevStage {
  static constexpr int kK = 0;
  static constexpr int kQ = BOTH ? TokenTile<NP, KS>::kBytes : 0;  // else Q takes K's place after it
  static constexpr int kTt = kQ + TokenTile<NP, KS>::kBytes;
  static constexpr int kPt = kTt + kTriBytes;
  static constexpr int kGates = kPt + kTriBytes;
  static constexpr int kdO = kGates + kGateFloats * 4;  // (64, kBlockCols) of InT
  static constexpr int kBytes = kdO + kChunk * kBlockCols * static_cast<int>(sizeof(InT));
};

template <typename InT>
struct RevSource {
  const InT* q;
  const InT* k;
  const InT* dout;  // the chunk's first token, column 0 of the head
  const char* record;
  int n_tokens;
};

struct RevOffsets {
  uint32_t k, q, o[2];
};

__device__ __forceinline__ RevOffsets rev_offsets(const ChunkArgs& a, int n_tokens, int col0, int lane, int wave) {
  RevOffsets o;
  const int last = n_tokens - 1, row = min(wave * 16 + (swizzled(lane) & 15), last);
  o.k = static_cast<uint32_t>(row) * static_cast<uint32_t>(a.ks) * 2 + (lane >> 4) * 16;
  o.q = static_cast<uint32_t>(row) * static_cast<uint32_t>(a.qs) * 2 + (lane >> 4) * 16;
  const int col = min(col0 + (lane & 7) * 8, a.dv - 8);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    o.o[i] = static_cast<uint32_t>(min((wave * 2 + i) * 8 + lane / 8, last)) * static_cast<uint32_t>(a.Hv * a.dv) * 2 + col * 2;
  return o;
}

// Straight into LDS; rows past the end repeat the last token (masked when used).
template <typename InT, int KS>
__device__ __forceinline__ void rev_stage_async(char* st, const RevSource<InT>& s, const RevOffsets& o, int lane,
                                                int wave) {
  using S = RevStage<InT, 1, KS, true>;
  const char *k = reinterpret_cast<const char*>(s.k), *q = reinterpret_cast<const char*>(s.q);
  const char* d = reinterpret_cast<const char*>(s.dout);
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    load_to_lds(k + i * 64 + o.k, st + S::kK + (wave * KS + i) * 1024);
    load_to_lds(q + i * 64 + o.q, st + S::kQ + (wave * KS + i) * 1024);
  }
  constexpr int kRec = (2 * kTriBytes + kGateFloats * 4) / 1024;  // T^T, P^T and the scalars follow each other
#pragma unroll
  for (int i = 0; i < (kRec + kWaves - 1) / kWaves; ++i) {
    const int f = wave + i * kWaves;
    if (f < kRec) load_to_lds(s.record + kRecTt + f * 1024 + static_cast<uint32_t>(lane * 16), st + S::kTt + f * 1024);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) load_to_lds(d + o.o[i], st + S::kdO + (wave * 2 + i) * 1024);
}

template <typename InT, int NP, int KS, bool BOTH>
__device__ __forceinline__ void rev_stage_sync(char* st, const ChunkArgs& a, const RevSource<InT>& s, int col0) {
  using S = RevStage<InT, NP, KS, BOTH>;
  uint16_t* sk = reinterpret_cast<uint16_t*>(st + S::kK);
  uint16_t* sq = reinterpret_cast<uint16_t*>(st + S::kQ);
  stage_rows<InT, NP, KS, kThreads>(sk, s.k, a.ks, s.n_tokens, a.dk, a.vec);
  if constexpr (BOTH) stage_rows<InT, NP, KS, kThreads>(sq, s.q, a.qs, s.n_tokens, a.dk, a.vec);
  constexpr int kRuns = (2 * kTriBytes + kGateFloats * 4) / 16;
  for (int i = threadIdx.x; i < kRuns; i += kThreads)
    reinterpret_cast<u32x4*>(st + S::kTt)[i] = reinterpret_cast<const u32x4*>(s.record + kRecTt)[i];
  InT* o = reinterpret_cast<InT*>(st + S::kdO);
#pragma unroll
  for (int i = 0; i < kChunk * kBlockCols / kThreads; ++i) {
    const int e = threadIdx.x + i * kThreads, token = e / kBlockCols, col = col0 + e % kBlockCols;
    InT x{};
    if (token < s.n_tokens && col < a.dv) x = s.dout[static_cast<int64_t>(token) * a.Hv * a.dv + col];
    o[e] = x;
  }
}

// The walk from the last chunk to the first: 16 columns of dH a wave, as in the forward,
//   dU = P^T dO + eC (K dH1),  dR = T^T dU,  dV = beta dR,
//   dH0 = aC dH1 + Q^T (e0 dO) - K^T (beta e0 dR).
// On few heads it goes in the forward's pieces: a first pass finds what every piece adds to
// dH at its start, the fold carries dH back over them by the transposes of the forward's M,
// and the full pass starts every piece from its own dH (1 x 4096 x 2 heads: the
// whole backward 489 us without, 215 with; this kernel 21 us for the first pass, 35 for the second).
// Bound like the forward's walk by the chain of a chunk's products, one wave a SIMD, and
// it writes dH1 and dR for the gradients' kernel besides: 260 us for 8 x 2048 x 12 heads of
// 128 x 128 (1.8 TB/s), against 186 for the walk that leaves H0 and U.
template <typename InT, int NP, int KS, bool BOTH, bool ASYNC, int STAGES>
__global__ __launch_bounds__(kThreads) void delta_chunk_reverse(const BwdArgs s) {
  using Tile = TokenTile<NP, KS>;
  using S = RevStage<InT, NP, KS, BOTH>;
  constexpr int DKT = 2 * KS;
  extern __shared__ __align__(16) char staged[];
  const ChunkArgs& a = s.c;
  const int lane = threadIdx.x % 64, wave = wave_index(), g4 = (lane >> 4) * 4;
  const Place place = place_of(blockIdx.x, s.col_blocks);
  const int cb = place.part, bh = place.item / s.pieces, piece = place.item - bh * s.pieces;
  if (bh >= s.heads) return;
  const int c0 = piece * s.chunks_piece, c1 = min(a.chunks, c0 + s.chunks_piece);
  const bool all = s.agg == nullptr;
  const int b = bh / a.Hv, h = bh - b * a.Hv, hk = h / a.group;
  const int col0 = cb * kBlockCols, own = col0 + wave * 16 + (lane & 15);
  const bool has_v = own < a.dv;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

  f32x4 H[DKT];  // dH
#pragma unroll
  for (int m = 0; m < DKT; ++m) {
    H[m] = zero;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = state_row(m, g4, r);
      if (!all) continue;
      if (piece + 1 < s.pieces) {
        if (own < s.cols)
          H[m][r] = s.ends[((static_cast<int64_t>(bh) * s.pieces + piece) * (32 * KS) + row) * s.cols + own];
      } else if (s.dh_last && row < a.dk && has_v) {
        H[m][r] = s.dh_last[(static_cast<int64_t>(bh) * a.dk + row) * a.dv + own];
      }
    }
  }
  const int64_t token_v = static_cast<int64_t>(a.Hv) * a.dv;
  RevSource<InT> src;
  {
    const int64_t t0 = static_cast<int64_t>(b) * a.L + static_cast<int64_t>(c1 - 1) * kChunk;
    src.q = static_cast<const InT*>(a.q) + t0 * a.qs + static_cast<int64_t>(hk) * a.dk;
    src.k = static_cast<const InT*>(a.k) + t0 * a.ks + static_cast<int64_t>(hk) * a.dk;
    src.dout = static_cast<const InT*>(s.dout) + t0 * token_v + static_cast<int64_t>(h) * a.dv;
    src.record = a.records + (static_cast<int64_t>(bh) * a.chunks + c1 - 1) * kRecBytesBwd;
    src.n_tokens = static_cast<int>(min(static_cast<int64_t>(kChunk), a.L - static_cast<int64_t>(c1 - 1) * kChunk));
  }
  const RevOffsets whole = rev_offsets(a, kChunk, col0, lane, wave);
  const auto stage = [&](char* st, const RevSource<InT>& from) {
    if constexpr (ASYNC)
      rev_stage_async<InT, KS>(st, from,
                               from.n_tokens == kChunk ? whole : rev_offsets(a, from.n_tokens, col0, lane, wave), lane,
                               wave);
    else
      rev_stage_sync<InT, NP, KS, BOTH>(st, a, from, col0);
  };
  if constexpr (STAGES == 2) stage(staged, src);
  for (int c = c1 - 1; c >= c0; --c) {
    char* st = staged + (STAGES == 2 ? ((c1 - 1 - c) & 1) * S::kBytes : 0);
    RevSource<InT> next = src;
    next.q -= kChunk * a.qs;
    next.k -= kChunk * a.ks;
    next.dout -= kChunk * token_v;
    next.record -= kRecBytesBwd;
    next.n_tokens = kChunk;
    if constexpr (STAGES == 2) {
      wait_loads();
      __syncthreads();  // this stage is loaded, and the other one is no longer read
      if (c > c0) stage(staged + ((c1 - c) & 1) * S::kBytes, next);
    } else {
      __syncthreads();  // the previous chunk is no longer read
      stage(st, src);
      wait_loads();
      __syncthreads();
    }
    const uint16_t* sk = reinterpret_cast<const uint16_t*>(st + S::kK);
    const uint16_t* sq = reinterpret_cast<const uint16_t*>(st + S::kQ);
    const float* gates = reinterpret_cast<const float*>(st + S::kGates);
    const int64_t record = static_cast<int64_t>(bh) * a.chunks + c;

    if (all && own < s.cols) {
      float* to = s.dstates + record * (32 * KS) * s.cols + own;
#pragma unroll
      for (int m = 0; m < DKT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) to[static_cast<int64_t>(state_row(m, g4, r)) * s.cols] = H[m][r];
    }

    // K dH1, and the lane's column of dO
    f32x4 X[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Frag<3> hb = split8(H[2 * ks], H[2 * ks + 1]);
      Frag<NP> kf[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) kf[m] = Tile::rows(sk, m, ks, lane);
      mma_n(kf, hb, X);
    }
    f32x4 dO[4];
    Frag<NP> ob[2];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if constexpr (sizeof(InT) == 2) {
        u32x2 w = read_transposed(reinterpret_cast<const uint16_t*>(st + S::kdO) +
                                  (m * 16 + g4 + ((lane & 15) >> 2)) * kBlockCols + wave * 16 + (lane & 3) * 4);
        if (src.n_tokens < kChunk) {
          const int left = src.n_tokens - (m * 16 + g4);  // tokens of the four that exist
          w.x = left >= 2 ? w.x : left == 1 ? w.x & 0xFFFFu : 0u;
          w.y = left >= 4 ? w.y : left == 3 ? w.y & 0xFFFFu : 0u;
        }
        dO[m] = f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                      __uint_as_float(w.y & 0xFFFF0000u)};
        if (m & 1) {
          ob[m / 2].p[0].z = w.x;
          ob[m / 2].p[0].w = w.y;
        } else {
          ob[m / 2].p[0].x = w.x;
          ob[m / 2].p[0].y = w.y;
        }
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          dO[m][r] = reinterpret_cast<const float*>(st + S::kdO)[(m * 16 + g4 + r) * kBlockCols + wave * 16 + (lane & 15)];
      }
    }
    if constexpr (NP == 3) {
      ob[0] = split8(dO[0], dO[1]);
      ob[1] = split8(dO[2], dO[3]);
    }
    f32x4 dU[4] = {zero, zero, zero, zero};
    mma_tri_t(reinterpret_cast<const uint16_t*>(st + S::kPt), ob, lane, dU);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const f32x4 eC = *reinterpret_cast<const f32x4*>(gates + kEC + m * 16 + g4);
#pragma unroll
      for (int r = 0; r < 4; ++r) dU[m][r] = __builtin_fmaf(eC[r], X[m][r], a.scale * dU[m][r]);
    }
    f32x4 dR[4] = {zero, zero, zero, zero};
    {
      const Frag<3> ub[2] = {split8(dU[0], dU[1]), split8(dU[2], dU[3])};
      mma_tri_t(reinterpret_cast<const uint16_t*>(st + S::kTt), ub, lane, dR);
    }
    if (all && own < s.cols) {
      float* to = s.dR + record * kChunk * s.cols + own;
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) to[(m * 16 + g4 + r) * s.cols] = dR[m][r];
    }
    const float aC = gates[kAC];
    f32x4 dV[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const f32x4 e0 = *reinterpret_cast<const f32x4*>(gates + kE0 + m * 16 + g4);
      const f32x4 be = *reinterpret_cast<const f32x4*>(gates + kBeta + m * 16 + g4);
      dV[m] = be * dR[m];
      dR[m] = -e0 * dV[m];
      dO[m] *= a.scale * e0;
    }
#pragma unroll
    for (int m = 0; m < DKT; ++m) H[m] *= aC;
    {
      const Frag<3> rb[2] = {split8(dR[0], dR[1]), split8(dR[2], dR[3])};
#pragma unroll
      for (int ts = 0; ts < 2; ++ts) {
        Frag<NP> kc[DKT];
#pragma unroll
        for (int m = 0; m < DKT; ++m) kc[m] = Tile::columns(sk, m, ts, lane);
        mma_n(kc, rb[ts], H);
      }
    }
    if constexpr (!BOTH) {
      __syncthreads();
      stage_rows<InT, NP, KS, kThreads>(reinterpret_cast<uint16_t*>(st + S::kQ), src.q, a.qs, src.n_tokens, a.dk, a.vec);
      __syncthreads();
    }
    {
      const Frag<3> qb[2] = {split8(dO[0], dO[1]), split8(dO[2], dO[3])};
#pragma unroll
      for (int ts = 0; ts < 2; ++ts) {
        Frag<NP> qc[DKT];
#pragma unroll
        for (int m = 0; m < DKT; ++m) qc[m] = Tile::columns(sq, m, ts, lane);
        mma_n(qc, qb[ts], H);
      }
    }

    const int64_t row0 = (static_cast<int64_t>(b) * a.L + static_cast<int64_t>(c) * kChunk) * a.Hv + h;  // x dv
    if (!all) {
      // the piece's start alone is wanted
    } else if (ASYNC && s.grad_bf16) {
      // turned to rows in the place of the strip's dO, as the forward's outputs
      uint16_t* o = reinterpret_cast<uint16_t*>(st + S::kdO) + wave * 16;
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          const uint32_t w = bf16_words(dV[m][r], dV[m][r + 1]);
          uint16_t* p = o + (m * 16 + g4 + r) * kBlockCols + (lane & 15);
          p[0] = static_cast<uint16_t>(w);
          p[kBlockCols] = static_cast<uint16_t>(w >> 16);
        }
      char* dst = static_cast<char*>(s.dv) + (row0 * a.dv + col0 + wave * 16) * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int token = i * 32 + lane / 2, half = (lane & 1) * 8;
        const u32x4 w = *reinterpret_cast<const u32x4*>(o + token * kBlockCols + half);
        if (token < src.n_tokens && col0 + wave * 16 + half < a.dv)
          *reinterpret_cast<u32x4*>(dst + static_cast<uint32_t>(token * a.Hv * a.dv + half) * 2) = w;
      }
    } else {
      const int64_t lane0 = row0 * a.dv + g4 * token_v + own;
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (!has_v || m * 16 + g4 + r >= src.n_tokens) continue;
          if (s.grad_bf16)
            store_elem(static_cast<bf16_t*>(s.dv) + (m * 16 + r) * token_v, lane0, dV[m][r]);
          else
            store_elem(static_cast<float*>(s.dv) + (m * 16 + r) * token_v, lane0, dV[m][r]);
        }
    }
    src = next;
  }
  if (!all) {
    const int width = 32 * KS + s.cols;
    float* to = s.agg + (static_cast<int64_t>(bh) * s.pieces + piece) * (32 * KS) * width + 32 * KS + own;
    if (own < s.cols) {
#pragma unroll
      for (int m = 0; m < DKT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) to[static_cast<int64_t>(state_row(m, g4, r)) * width] = H[m][r];
    }
  } else if (piece == 0 && s.dh0 && has_v) {
#pragma unroll
    for (int m = 0; m < DKT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = state_row(m, g4, r);
        if (row < a.dk) s.dh0[(static_cast<int64_t>(bh) * a.dk + row) * a.dv + own] = H[m][r];
      }
  }
}

// ---- the gradients of a chunk ----

// A workgroup takes up to 64 entries of q and k (SL tiles of 32; 96 where they are 65 to
// 96): its accumulators then come near 256 registers, and two workgroups share a CU, one multiplying while the other waits
// for its operands. P and S are made anew for every split. 8 x 2048 x 12 heads of 128 x 128:
// 548 us with all entries in one workgroup of eight waves, 417 so split, 360 with the
// staged tiles turned against bank conflicts and 32-bit offsets from uniform bases; its
// states, U, dR and dO are 0.65 GB (1.8 TB/s). Half of a wave's cycles are still waits:
// every slab of 32 columns is split into bfloat16 parts, stored and read back between two
// barriers. Every instance spills some of what it holds through the sums over dv: 13 to 57
// registers for bfloat16 (174 with 96 entries), 38 to 221 for float32, which is 240 MB written
// beside the results of that call. (Split by rows and columns of P instead: 1004 us, spilled.)
__host__ __device__ constexpr int split_tiles(int ks) { return ks % 2 == 0 ? 2 : ks == 3 ? 3 : 1; }
constexpr int grad_splits(int ks) { return ks / split_tiles(ks); }
// A split's sums: own, end, the diagonal of dR U^T (64 tokens each), <dH1, H0>.
constexpr int kSumOwn = 0, kSumEnd = 64, kSumBeta = 128, kSumState = 192, kSumFloats = 256;

// Tile row that a state row is staged at, so that column n of tile m is state_row(m, ..).
__device__ __forceinline__ int staged_row(int row) {
  return ((row >> 5) * 2 + ((row >> 2) & 1)) * 16 + ((row >> 3) & 3) * 4 + (row & 3);
}

// One thread's part of a 32-column slab: eight columns of one row of dO, U and dR, and of
// ITEMS rows of H0 and dH1.
template <int NP, int ITEMS>
struct SlabLoads {
  u32x4 o[NP == 1 ? 1 : 2];  // as they lie in memory
  f32x4 u[2], r[2], h[ITEMS][2], g[ITEMS][2];
};

template <int NP, int TILES>
__device__ __forceinline__ Frag<NP> slab_rows(const uint16_t* s, int tile, int lane) {
  Frag<NP> f;
#pragma unroll
  for (int k = 0; k < NP; ++k) f.p[k] = *reinterpret_cast<const u32x4*>(s + k * TILES * 512 + (tile * 64 + swizzled(lane)) * 8);
  return f;
}
template <int TILES>
__device__ __forceinline__ void store_slab(uint16_t* s, int at, int oct, const f32x4 (&x)[2]) {
  const Frag<3> f = split8(x[0], x[1]);
#pragma unroll
  for (int k = 0; k < 3; ++k)
    *reinterpret_cast<u32x4*>(s + k * TILES * 512 + ((at >> 4) * 64 + swizzled(oct * 16 + (at & 15))) * 8) = f.p[k];
}

// LDS of a workgroup: the slab, and its entries of the staged tokens of K and Q, beside it
// for the whole call where two workgroups still fit a CU, else in its place after each head.
template <int NP, int SL>
struct GradLds {
  static constexpr int kdO = 0;
  static constexpr int kU = kdO + NP * 4096;
  static constexpr int kdR = kU + 3 * 4096;
  static constexpr int kH = kdR + 3 * 4096;
  static constexpr int kdH = kH + 3 * 2 * SL * 1024;
  static constexpr int kSlab = kdH + 3 * 2 * SL * 1024;
  static constexpr int kTile = TokenTile<NP, SL>::kBytes;
  static constexpr bool kBeside = kSlab + 2 * kTile <= 76 * 1024;
  static constexpr int kK = kBeside ? kSlab : 0;
  static constexpr int kQ = kK + kTile;
  static constexpr int kBytes = kBeside ? kSlab + 2 * kTile : std::max(kSlab, 2 * kTile);
};

// The lane's column of the four tokens 16 w + g4 .. of a staged tile, from the operand
// that holds the tokens 32 (w / 2) ..
template <int NP>
__device__ __forceinline__ f32x4 column_values(const Frag<NP>& f, int w) {
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = NP - 1; i >= 0; --i) {
    const uint32_t lo = (w & 1) ? f.p[i].z : f.p[i].x, hi = (w & 1) ? f.p[i].w : f.p[i].y;
    v += f32x4{__uint_as_float(lo << 16), __uint_as_float(lo & 0xFFFF0000u), __uint_as_float(hi << 16),
               __uint_as_float(hi & 0xFFFF0000u)};
  }
  return v;
}

// Keeps the compiler from reading the operands of many tiles ahead, which spills.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// One workgroup: 32 SL entries of a chunk of one key head, its value heads in turn; wave w
// has the tokens of tile w as rows of dQ and dK. The sums over dv go in slabs of 32
// columns, the next one's loads under way while one is multiplied.
// VEC: rows of dout come as whole 16-byte runs.
template <typename InT, int NP, int SL, bool VEC>
__global__ __launch_bounds__(kThreads, 2) void delta_chunk_grads(const BwdArgs s, int splits) {
  using Lds = GradLds<NP, SL>;
  using Tile = TokenTile<NP, SL>;
  constexpr int MT = 2 * SL, ROWS = 32 * SL, ITEMS = ROWS * 4 / kThreads > 0 ? (ROWS * 4 + kThreads - 1) / kThreads : 1;
  extern __shared__ __align__(16) char staged[];
  __shared__ __align__(16) float scalars[kGateFloatsBwd];
  __shared__ __align__(16) float diag_dP[64], waves_sum[kWaves];
  const ChunkArgs& a = s.c;
  const int lane = threadIdx.x % 64, w = wave_index();
  const int g4 = (lane >> 4) * 4, col = lane & 15;
  const Place place = place_of(blockIdx.x, splits);  // the splits of a chunk read the same U, dR and dO
  const int split = place.part, item = place.item;
  if (item >= s.items) return;
  const int chunk = item % a.chunks, bhk = item / a.chunks;
  const int b = bhk / a.Hk, hk = bhk - b * a.Hk;
  const int first = split * ROWS, all_rows = splits * ROWS;  // the workgroup's entries, and the states' rows
  const int64_t t0 = static_cast<int64_t>(b) * a.L + static_cast<int64_t>(chunk) * kChunk;
  const int n_tokens = static_cast<int>(min(static_cast<int64_t>(kChunk), a.L - static_cast<int64_t>(chunk) * kChunk));
  const InT* q = static_cast<const InT*>(a.q) + t0 * a.qs + static_cast<int64_t>(hk) * a.dk + first;
  const InT* k = static_cast<const InT*>(a.k) + t0 * a.ks + static_cast<int64_t>(hk) * a.dk + first;
  uint16_t* sdO = reinterpret_cast<uint16_t*>(staged + Lds::kdO);
  uint16_t* sU = reinterpret_cast<uint16_t*>(staged + Lds::kU);
  uint16_t* sdR = reinterpret_cast<uint16_t*>(staged + Lds::kdR);
  uint16_t* sH = reinterpret_cast<uint16_t*>(staged + Lds::kH);
  uint16_t* sdH = reinterpret_cast<uint16_t*>(staged + Lds::kdH);
  uint16_t* sk = reinterpret_cast<uint16_t*>(staged + Lds::kK);
  uint16_t* sq = reinterpret_cast<uint16_t*>(staged + Lds::kQ);
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  // columns at or past dv (rounded up to 8) may hold copies of others: read as 0
  const int limit = (a.dv + 7) / 8 * 8;
  const int64_t token_v = static_cast<int64_t>(a.Hv) * a.dv;
  const int oct = threadIdx.x & 3, row = threadIdx.x >> 2;  // this thread's rows and columns of a slab
  const auto stage_qk = [&]() {
    stage_rows<InT, NP, SL, kThreads>(sk, k, a.ks, n_tokens, a.dk - first, a.vec);
    stage_rows<InT, NP, SL, kThreads>(sq, q, a.qs, n_tokens, a.dk - first, a.vec);
  };
  if constexpr (Lds::kBeside) stage_qk();

  f32x4 dq_sum[MT], dk_sum[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) dq_sum[m] = dk_sum[m] = zero;

  for (int gi = 0; gi < a.group; ++gi) {
    const int h = hk * a.group + gi, bh = b * a.Hv + h;
    const int64_t record = static_cast<int64_t>(bh) * a.chunks + chunk;
    const char* H0 = reinterpret_cast<const char*>(s.states + (record * all_rows + first) * s.cols);
    const char* dH1 = reinterpret_cast<const char*>(s.dstates + (record * all_rows + first) * s.cols);
    const char* U = reinterpret_cast<const char*>(s.U + record * kChunk * s.cols);
    const char* dR = reinterpret_cast<const char*>(s.dR + record * kChunk * s.cols);
    const InT* dout_first = static_cast<const InT*>(s.dout) + (t0 * a.Hv + h) * a.dv;
    const InT* dout = dout_first + row * token_v;
    const auto fetch = [&](SlabLoads<NP, ITEMS>& x, int d0) {
      const int c = d0 + oct * 8, from = c < limit ? c : 0;
      const uint32_t at = static_cast<uint32_t>(row * s.cols + from) * 4;  // bytes from a uniform base
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x.u[i] = *reinterpret_cast<const f32x4*>(U + at + 16 * i);
        x.r[i] = *reinterpret_cast<const f32x4*>(dR + at + 16 * i);
      }
#pragma unroll
      for (int n = 0; n < ITEMS; ++n) {
        const uint32_t at = static_cast<uint32_t>(min(row + n * (kThreads / 4), ROWS - 1) * s.cols + from) * 4;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          x.h[n][i] = *reinterpret_cast<const f32x4*>(H0 + at + 16 * i);
          x.g[n][i] = *reinterpret_cast<const f32x4*>(dH1 + at + 16 * i);
        }
      }
      const int left = row < n_tokens ? a.dv - c : 0;
      if constexpr (VEC) {
        const u32x4* o = reinterpret_cast<const u32x4*>(left > 0 ? dout + c : dout_first);
#pragma unroll
        for (int i = 0; i < (NP == 1 ? 1 : 2); ++i) x.o[i] = o[i];
      } else if constexpr (NP == 1) {
        uint32_t e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = j < left ? dout[c + j].bits : 0u;
        x.o[0] = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x.o[j / 4][j % 4] = j < left ? __float_as_uint(dout[c + j]) : 0u;
      }
    };
    SlabLoads<NP, ITEMS> loads;
    fetch(loads, 0);
    __syncthreads();  // the previous head's scalars are used
#pragma unroll
    for (int i = 0; i < kGateFloatsBwd / kThreads; ++i)
      scalars[i * kThreads + threadIdx.x] =
          reinterpret_cast<const float*>(a.records + record * kRecBytesBwd + kRecGatesBwd)[i * kThreads + threadIdx.x];

    f32x4 E1[MT], E2[MT], E3[MT];  // dO H0^T, dR H0^T, U dH1^T: rows of tile w, columns of the state tiles
#pragma unroll
    for (int m = 0; m < MT; ++m) E1[m] = E2[m] = E3[m] = zero;
    // Columns of tile w: rows of tile j < w of U dO^T and U dR^T, rows of tile j >= w of dO U^T
    // and dR U^T; and, apart, tile w of the first two
    f32x4 P[4] = {zero, zero, zero, zero}, S[4] = {zero, zero, zero, zero}, Pw = zero, Sw = zero;
    float hh = 0.0f;  // the thread's part of <dH1, H0>
#pragma unroll 1
    for (int d0 = 0; d0 < a.dv; d0 += 32) {
      __syncthreads();  // the last slab is read, or the previous head's tiles
      // Rows past the chunk's and columns past the head's were loaded from the first ones.
      const bool inside = d0 + oct * 8 < limit;
      if (!inside || row >= n_tokens) {
        for (u32x4& x : loads.o) x = u32x4{0, 0, 0, 0};
      }
      if (!inside) {
        loads.u[0] = loads.u[1] = loads.r[0] = loads.r[1] = zero;
#pragma unroll
        for (int n = 0; n < ITEMS; ++n) loads.h[n][0] = loads.h[n][1] = loads.g[n][0] = loads.g[n][1] = zero;
      }
      uint16_t* to = sdO + ((row >> 4) * 64 + swizzled(oct * 16 + (row & 15))) * 8;
      if constexpr (NP == 1) {
        *reinterpret_cast<u32x4*>(to) = loads.o[0];
      } else {
        const Frag<3> f = split8(__builtin_bit_cast(f32x4, loads.o[0]), __builtin_bit_cast(f32x4, loads.o[1]));
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<u32x4*>(to + i * 2048) = f.p[i];
      }
      store_slab<4>(sU, row, oct, loads.u);
      store_slab<4>(sdR, row, oct, loads.r);
#pragma unroll
      for (int n = 0; n < ITEMS; ++n) {
        const int r = row + n * (kThreads / 4);
        if (r < ROWS) {
          store_slab<MT>(sH, staged_row(r), oct, loads.h[n]);
          store_slab<MT>(sdH, staged_row(r), oct, loads.g[n]);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) hh = __builtin_fmaf(loads.h[n][i][j], loads.g[n][i][j], hh);
        }
      }
      if (d0 + 32 < a.dv) fetch(loads, d0 + 32);
      __syncthreads();
      const Frag<NP> dOw = slab_rows<NP, 4>(sdO, w, lane);
      const Frag<3> Uw = slab_rows<3, 4>(sU, w, lane), dRw = slab_rows<3, 4>(sdR, w, lane);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const Frag<3> hb = slab_rows<3, MT>(sH, m, lane), gb = slab_rows<3, MT>(sdH, m, lane);
        E1[m] = mma(dOw, hb, E1[m]);
        mma_pair(dRw, hb, E2[m], Uw, gb, E3[m]);
        keep_order();
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < w) {
          const Frag<3> Uj = slab_rows<3, 4>(sU, j, lane);
          P[j] = mma(Uj, dOw, P[j]);
          S[j] = mma(Uj, dRw, S[j]);
        } else {
          P[j] = mma(slab_rows<NP, 4>(sdO, j, lane), Uw, P[j]);
          S[j] = mma(slab_rows<3, 4>(sdR, j, lane), Uw, S[j]);
        }
        keep_order();
      }
      Pw = mma(Uw, dOw, Pw);
      Sw = mma(Uw, dRw, Sw);
    }

    // d beta comes from the diagonal of dR U^T, and dP's is set aside; then the decays and masks.
    float* sums = s.sums + (record * splits + split) * kSumFloats;
    const ColDecay cw = col_decay(scalars, w * 16 + col);
    if ((col >> 2) == (lane >> 4)) {
      const int r = col & 3;
      sums[kSumBeta + w * 16 + col] = r == 0 ? Sw.x : r == 1 ? Sw.y : r == 2 ? Sw.z : Sw.w;
      diag_dP[w * 16 + col] = a.scale * (r == 0 ? Pw.x : r == 1 ? Pw.y : r == 2 ? Pw.z : Pw.w);
    }
    // of rows of tile j: those before the columns (up), and those after them, which stay in P and S
    f32x4 Pc[4], Sc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const RowDecay rows = row_decay(scalars, j * 16 + g4);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int x = j * 16 + g4 + r, y = w * 16 + col;
        const float up = x < y ? decay_up(rows, r, cw) : 0.0f, down = x > y ? decay_down(rows, r, cw) : 0.0f;
        Pc[j][r] = (j == w ? Pw[r] : P[j][r]) * (a.scale * up);
        Sc[j][r] = (j == w ? Sw[r] : S[j][r]) * (-cw.beta * up);
        P[j][r] *= a.scale * down;
        S[j][r] *= -rows.beta[r] * down;
      }
    }
    const f32x4 e0 = *reinterpret_cast<const f32x4*>(scalars + kE0 + w * 16 + g4);
    const f32x4 eC = *reinterpret_cast<const f32x4*>(scalars + kEC + w * 16 + g4);
    const f32x4 be = *reinterpret_cast<const f32x4*>(scalars + kBeta + w * 16 + g4);
    // of the lane's four tokens, its columns' part: q . dq + k . (i side - j side), and k . eC (U dH1^T)
    f32x4 own = zero, ku = zero;
    __syncthreads();  // the slab is read, the diagonal is set
    if constexpr (!Lds::kBeside) {
      stage_qk();
      __syncthreads();
    }
    const f32x4 dp = *reinterpret_cast<const f32x4*>(&diag_dP[w * 16 + g4]);
    {  // what the tokens take from those before them, and the state's end
      const Frag<3> ap[2] = {split8(Pc[0], Pc[1]), split8(Pc[2], Pc[3])};
      const Frag<3> as[2] = {split8(Sc[0], Sc[1]), split8(Sc[2], Sc[3])};
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        E1[m] *= a.scale * e0;
        E2[m] *= -be * e0;
        E3[m] *= eC;
        f32x4 kv = zero, qv = zero;
#pragma unroll
        for (int ts = 0; ts < 2; ++ts) {
          if (ts > w / 2) continue;
          const Frag<NP> kc = Tile::columns(sk, m, ts, lane);
          if (ts == w / 2) {
            kv = column_values(kc, w);
            qv = column_values(Tile::columns(sq, m, ts, lane), w);
          }
          mma_pair(ap[ts], kc, E1[m], as[ts], kc, E2[m]);
        }
        ku += kv * E3[m];
        own += qv * E1[m] + kv * E2[m];
        dq_sum[m] += E1[m] + dp * kv;
        dk_sum[m] += (E2[m] + E3[m]) + dp * qv;
        keep_order();
      }
    }
    {  // what they give to those after them
      const Frag<3> bp[2] = {split8(P[0], P[1]), split8(P[2], P[3])};
      const Frag<3> bs[2] = {split8(S[0], S[1]), split8(S[2], S[3])};
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 x = zero, y = zero, kv = zero;
#pragma unroll
        for (int ts = 0; ts < 2; ++ts) {
          if (ts < w / 2) continue;
          const Frag<NP> kc = Tile::columns(sk, m, ts, lane);
          if (ts == w / 2) kv = column_values(kc, w);
          mma_pair(bs[ts], kc, x, bp[ts], Tile::columns(sq, m, ts, lane), y);
        }
        own -= kv * (x + y);
        dk_sum[m] += x + y;
        keep_order();
      }
    }
    // sums over the 16 columns' lanes, and over the workgroup
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      own[r] = lanes_sum<16>(own[r]);
      ku[r] = lanes_sum<16>(ku[r]);
    }
    if (col == 0) {
      *reinterpret_cast<f32x4*>(&sums[kSumOwn + w * 16 + g4]) = own;
      *reinterpret_cast<f32x4*>(&sums[kSumEnd + w * 16 + g4]) = ku;
    }
    const float total = lanes_sum<64>(hh);
    if (lane == 0) waves_sum[w] = total;
    __syncthreads();
    if (threadIdx.x == 0) sums[kSumState] = (waves_sum[0] + waves_sum[1]) + (waves_sum[2] + waves_sum[3]);
  }

  const int64_t token_k = static_cast<int64_t>(a.Hk) * a.dk;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int d = first + state_row(m, col & 12, col & 3);
    if (d >= a.dk) continue;
    const int64_t at = (t0 + w * 16 + g4) * token_k + static_cast<int64_t>(hk) * a.dk + d;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (w * 16 + g4 + r >= n_tokens) continue;
      if (s.grad_bf16) {
        store_elem(static_cast<bf16_t*>(s.dq) + r * token_k, at, dq_sum[m][r]);
        store_elem(static_cast<bf16_t*>(s.dk) + r * token_k, at, dk_sum[m][r]);
      } else {
        store_elem(static_cast<float*>(s.dq) + r * token_k, at, dq_sum[m][r]);
        store_elem(static_cast<float*>(s.dk) + r * token_k, at, dk_sum[m][r]);
      }
    }
  }
}

// The gates' gradients: a wave for a chunk of a value head, a lane per token.
template <typename InT>
__global__ __launch_bounds__(kThreads) void delta_gate_grads(const BwdArgs s, int splits, int64_t records) {
  const ChunkArgs& a = s.c;
  const int lane = threadIdx.x % 64;
  const int64_t record = static_cast<int64_t>(blockIdx.x) * kWaves + wave_index();
  if (record >= records) return;
  const int bh = static_cast<int>(record / a.chunks), chunk = static_cast<int>(record - static_cast<int64_t>(bh) * a.chunks);
  const int b = bh / a.Hv, h = bh - b * a.Hv;
  const int n_tokens = static_cast<int>(min(static_cast<int64_t>(kChunk), a.L - static_cast<int64_t>(chunk) * kChunk));
  const float* scalars = reinterpret_cast<const float*>(a.records + record * kRecBytesBwd + kRecGatesBwd);
  const float* sums = s.sums + record * splits * kSumFloats;
  double from = 0.0, end = 0.0, state = 0.0;
  for (int i = 0; i < splits; ++i) {
    from += sums[i * kSumFloats + kSumOwn + lane];
    end += sums[i * kSumFloats + kSumEnd + lane];
    state += sums[i * kSumFloats + kSumState];
  }
  // sums within the token's document: from it on, and (eC is 0 before the last document) up to it
  const float seg = scalars[kSeg + lane];
  double upto = end;
#pragma unroll
  for (int off = 1; off < 64; off *= 2) {
    const double after = __shfl_down(from, off), before = __shfl_up(upto, off);
    const float seg_after = __shfl_down(seg, off), seg_up = __shfl_up(seg, off);
    if (lane + off < 64 && seg_after == seg) from += after;
    if (lane >= off && seg_up == seg) upto += before;
  }
  const double sum = from + (upto - end) + scalars[kAC] * state;
  const float seg_before = __shfl_up(seg, 1);
  const bool cut = lane == 0 ? seg > 0.0f : seg != seg_before;
  const bool there = lane < n_tokens;
  // nothing crosses a document's start: its token's gate has no part in the sums, whatever it is
  const bool off = cut || !there;
  const float dg = off ? 0.0f : static_cast<float>(sum);
  const float d_dt = off ? 0.0f : dg * a.A[h] * scalars[kSlope + lane];
  if (there) {
    const int64_t at = (static_cast<int64_t>(b) * a.L + static_cast<int64_t>(chunk) * kChunk + lane) * a.Hv + h;
    // 1 - beta / beta_scale is the sigmoid of -beta_raw, of which a beta near its limit keeps nothing
    const float rest = fast_rcp(1.0f + fast_exp2(load_elem(static_cast<const InT*>(a.br), at) * kLog2e));
    const float d_beta = sums[kSumBeta + lane] * rest;
    if (s.grad_bf16) {
      store_elem(static_cast<bf16_t*>(s.ddt), at, d_dt);
      store_elem(static_cast<bf16_t*>(s.dbr), at, d_beta);
    } else {
      store_elem(static_cast<float*>(s.ddt), at, d_dt);
      store_elem(static_cast<float*>(s.dbr), at, d_beta);
    }
  }
  const float dA = lanes_sum<64>(off ? 0.0f : dg * scalars[kDelta + lane]), dbias = lanes_sum<64>(d_dt);
  if (lane == 0) {
    s.part[record * 2] = dA;
    s.part[record * 2 + 1] = dbias;
  }
}

// dA and d dt_bias of a head: its chunks' parts over all batch rows, in a fixed order.
__global__ __launch_bounds__(kThreads) void delta_head_sums(const float* __restrict__ part, float* dA, float* dbias,
                                                            int B, int Hv, int chunks) {
  __shared__ float2 t[kThreads];
  const int h = blockIdx.x;
  const int64_t n = static_cast<int64_t>(B) * chunks;
  float2 x = make_float2(0.0f, 0.0f);
  for (int64_t i = threadIdx.x; i < n; i += kThreads) {
    const int64_t b = i / chunks, c = i - b * chunks;
    const float* p = part + ((b * Hv + h) * chunks + c) * 2;
    x.x += p[0];
    x.y += p[1];
  }
  t[threadIdx.x] = x;
  for (int off = kThreads / 2; off > 0; off /= 2) {
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < off) {
      t[threadIdx.x].x += t[threadIdx.x + off].x;
      t[threadIdx.x].y += t[threadIdx.x + off].y;
    }
  }
  if (threadIdx.x == 0) {
    dA[h] = t[0].x;
    if (dbias) dbias[h] = t[0].y;
  }
}

template <typename InT, int NP, int KS, bool ASYNC>
hipError_t launch_reverse(const BwdArgs& s, hipStream_t stream) {
  constexpr bool BOTH = RevStage<InT, NP, KS, true>::kBytes <= kMaxLds;
  constexpr int kBytes = RevStage<InT, NP, KS, BOTH>::kBytes;
  constexpr int STAGES = ASYNC && 2 * kBytes <= kMaxLds ? 2 : 1;
  static_assert(kBytes <= kMaxLds && (BOTH || !ASYNC), "a chunk's stage exceeds LDS");
  const int64_t blocks = placed_blocks(static_cast<int64_t>(s.heads) * s.pieces, s.col_blocks);
  SSM_LOG("launch delta_chunk_reverse<%d parts, %d rows>: %d chunks, %d stages of %d bytes; grid %lld x %d threads", NP,
          32 * KS, s.c.chunks, STAGES, kBytes, static_cast<long long>(blocks), kThreads);
  hipLaunchKernelGGL((delta_chunk_reverse<InT, NP, KS, BOTH, ASYNC, STAGES>), dim3(static_cast<unsigned>(blocks)),
                     dim3(kThreads), STAGES * kBytes, stream, s);
  return hipGetLastError();
}

template <typename InT, int NP, int KS>
hipError_t launch_grads(const BwdArgs& s, int64_t B, hipStream_t stream) {
  constexpr int SL = split_tiles(KS), splits = grad_splits(KS);
  constexpr int kBytes = GradLds<NP, SL>::kBytes;
  static_assert(kBytes + 4096 <= kMaxLds, "a slab exceeds LDS");
  const int64_t blocks = placed_blocks(s.items, splits);
  SSM_LOG("launch delta_chunk_grads<%d parts, %d entries>: %d splits; grid %lld x %d threads", NP, 32 * SL, splits,
          static_cast<long long>(blocks), kThreads);
  const dim3 grid_dim(static_cast<unsigned>(blocks));
  if (s.vec_out)
    hipLaunchKernelGGL((delta_chunk_grads<InT, NP, SL, true>), grid_dim, dim3(kThreads), kBytes, stream, s, splits);
  else
    hipLaunchKernelGGL((delta_chunk_grads<InT, NP, SL, false>), grid_dim, dim3(kThreads), kBytes, stream, s, splits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t records = B * s.c.Hv * s.c.chunks, grid = (records + kWaves - 1) / kWaves;
  SSM_LOG("launch delta_gate_grads: grid %lld x %d threads", static_cast<long long>(grid), kThreads);
  hipLaunchKernelGGL((delta_gate_grads<InT>), dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, s, splits,
                     records);
  return hipGetLastError();
}

struct Pieces {  // what the fold between the reverse walks needs
  const DeltaPlan& p;
  const DeltaChunks& plan;
  char* ws;
  float* agg;
};

template <typename InT, int NP, int KS>
hipError_t launch_both(const BwdArgs& s, const Pieces& cut, bool direct, hipStream_t stream) {
  const auto reverse = [&](const BwdArgs& args) {
    if constexpr (NP == 1)
      if (direct) return launch_reverse<InT, NP, KS, true>(args, stream);
    return launch_reverse<InT, NP, KS, false>(args, stream);
  };
  hipError_t e;
  if (s.pieces > 1) {
    BwdArgs ends = s;
    ends.agg = cut.agg;
    if ((e = reverse(ends)) != hipSuccess) return e;
    if ((e = launch_delta_fold_back(cut.p, cut.plan, cut.ws, s.dh_last, stream)) != hipSuccess) return e;
  }
  e = reverse(s);
  return e == hipSuccess ? launch_grads<InT, NP, KS>(s, cut.p.B, stream) : e;
}

template <typename InT, int NP>
hipError_t launch_ks(const BwdArgs& s, const Pieces& cut, bool direct, hipStream_t stream) {
  switch (padded_ks(s.c.dk)) {
    case 1: return launch_both<InT, NP, 1>(s, cut, direct, stream);
    case 2: return launch_both<InT, NP, 2>(s, cut, direct, stream);
    case 3: return launch_both<InT, NP, 3>(s, cut, direct, stream);
    case 4: return launch_both<InT, NP, 4>(s, cut, direct, stream);
    case 6: return launch_both<InT, NP, 6>(s, cut, direct, stream);
    default: return launch_both<InT, NP, 8>(s, cut, direct, stream);
  }
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

DeltaBwdLayout plan_delta_bwd(int64_t B, int64_t L, int Hv, int dk, int dv) {
  DeltaBwdLayout d{};
  d.chunks = static_cast<int>((L + kChunk - 1) / kChunk);
  const size_t n = static_cast<size_t>(B) * Hv * d.chunks;
  const size_t rows = 32 * static_cast<size_t>(padded_ks(dk)), cols = (static_cast<size_t>(dv) + 15) / 16 * 16;
  size_t off = 0;
  const auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  d.off_records = take(n * kRecBytesBwd);
  d.off_states = take(n * rows * cols * 4);
  d.off_U = take(n * kChunk * cols * 4);
  d.off_dstates = take(n * rows * cols * 4);
  d.off_dR = take(n * kChunk * cols * 4);
  d.off_sums = take(n * grad_splits(padded_ks(dk)) * kSumFloats * 4);
  d.off_part = take(n * 2 * 4);
  // the forward's pieces, behind the records that they have here
  d.walk = plan_delta_chunks(B, L, Hv, dk, dv, 0);
  const size_t records = d.walk.off_agg, at = take(d.walk.bytes - records);
  for (size_t* o : {&d.walk.off_agg, &d.walk.off_starts, &d.walk.off_group_agg, &d.walk.off_group_starts})
    *o += at - records;
  if (d.walk.pieces > 1) d.walk.off_turned = take(static_cast<size_t>(B) * Hv * d.walk.pieces * rows * rows * 4);
  d.bytes = off;
  return d;
}

bool delta_bwd_grids_fit(int64_t heads, int64_t key_heads, int dk, int dv, const DeltaBwdLayout& d) {
  return delta_grids_fit(heads, dk, dv, d.walk) &&
         fits_launch(placed_blocks(key_heads * d.chunks, grad_splits(padded_ks(dk))), kThreads);
}

hipError_t launch_delta_bwd(const DeltaPlan& p, const DeltaBwdPlan& g, const DeltaBwdLayout& lay, void* workspace,
                            hipStream_t stream) {
  char* ws = static_cast<char*>(workspace);
  BwdArgs s{};
  s.c = chunk_args(p, lay.chunks);
  s.c.records = ws + lay.off_records;
  hipError_t e = launch_chunk_prepare(p, s.c, true, stream);
  if (e != hipSuccess) return e;
  float* states = reinterpret_cast<float*>(ws + lay.off_states);
  float* U = reinterpret_cast<float*>(ws + lay.off_U);
  if ((e = launch_delta_states(p, s.c, lay.walk, ws, states, U, stream)) != hipSuccess) return e;
  s.states = states;
  s.U = U;
  s.dstates = reinterpret_cast<float*>(ws + lay.off_dstates);
  s.dR = reinterpret_cast<float*>(ws + lay.off_dR);
  s.sums = reinterpret_cast<float*>(ws + lay.off_sums);
  s.part = reinterpret_cast<float*>(ws + lay.off_part);
  s.heads = static_cast<int>(p.B * p.Hv);
  s.pieces = lay.walk.pieces;
  s.chunks_piece = lay.walk.chunks_piece;
  s.ends = reinterpret_cast<const float*>(ws + lay.walk.off_starts);
  const Pieces cut{p, lay.walk, ws, reinterpret_cast<float*>(ws + lay.walk.off_agg)};
  s.items = static_cast<int>(p.B * p.Hk * lay.chunks);
  s.cols = (p.dv + 15) / 16 * 16;
  s.col_blocks = (p.dv + kBlockCols - 1) / kBlockCols;
  s.grad_bf16 = g.grad_bf16;
  s.dout = g.dout;
  s.dh_last = g.dh_last;
  s.dq = g.dq;
  s.dk = g.dk;
  s.dv = g.dv;
  s.ddt = g.ddt;
  s.dbr = g.dbr;
  s.dh0 = g.dh0;
  const int64_t reach = int64_t{1} << 24;  // elements a token, for 32-bit offsets inside a chunk
  s.vec_out = p.dv % 8 == 0 && delta_aligned(g.dout, 16);
  const bool direct = s.c.vec && s.vec_out && p.in_bf16 && p.dk == 32 * padded_ks(p.dk) && p.qs < reach && p.ks < reach &&
                      static_cast<int64_t>(p.Hv) * p.dv < reach && delta_aligned(g.dv, 16);
  e = p.in_bf16 ? launch_ks<bf16_t, 1>(s, cut, direct, stream) : launch_ks<float, 3>(s, cut, false, stream);
  if (e != hipSuccess) return e;
  SSM_LOG("launch delta_head_sums: grid %d x %d threads", p.Hv, kThreads);
  hipLaunchKernelGGL(delta_head_sums, dim3(p.Hv), dim3(kThreads), 0, stream, s.part, g.dA, g.dbias,
                     static_cast<int>(p.B), p.Hv, lay.chunks);
  return hipGetLastError();
}

}  // namespace ssm
