// The walk over the chunks of a head (delta_chunk.hip tells the mathematics) and its
// launches. Each of delta_walk_*.hip instantiates them for one kind of staging.
#pragma once

#include <algorithm>

#include "delta_chunk.h"

namespace ssm {

// What a walk leaves: the outputs, a piece's effect on the state, or every chunk's
// first state and U (for the backward).
enum Walk { kOutputs, kAggregates, kStates };

struct ScanArgs {
  ChunkArgs c;
  int pieces, chunks_piece;
  int items;        // heads x pieces
  int col_blocks;   // workgroups per item
  int out_bf16, out_runs;  // out_runs: rows of out take whole 16-byte runs
  const float* h0;  // (bh, dk, dv) or null
  const float* starts;  // states of pieces 1 .. (bh, piece, 32 KS, cols), or null
  float* agg;       // aggregates walk: (bh, piece, 32 KS, 32 KS + cols)
  float* turned;    // M^T as well: (bh, piece, 32 KS, 32 KS), or null
  float* group_agg;     // of groups of pieces, as agg
  float* group_starts;  // and the states that they start from, as starts
  int cols;         // dv rounded up to 16
  void* out;
  float* h_last;
  float* states;    // states walk: (bh, chunk, 32 KS, cols)
  float* U;         // states walk: (bh, chunk, 64, cols)
  int64_t record_bytes, record_gates;
};

// The states that pieces 1 .. start from, from the aggregates (delta_chunk.hip).
hipError_t launch_delta_fold(const DeltaPlan& p, const DeltaChunks& plan, const ScanArgs& s, hipStream_t stream);
// The walks of a forward call, aggregates and fold included (one of delta_walk_*.hip each).
hipError_t launch_walk_bf16_direct(const DeltaPlan& p, const DeltaChunks& plan, const ScanArgs& s, hipStream_t stream);
hipError_t launch_walk_bf16(const DeltaPlan& p, const DeltaChunks& plan, const ScanArgs& s, hipStream_t stream);
hipError_t launch_walk_f32(const DeltaPlan& p, const DeltaChunks& plan, const ScanArgs& s, hipStream_t stream);

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kBlockCols = 16 * kWaves;  // columns of the state per workgroup

// What a workgroup stages of one chunk, in bytes from the stage's start. T, P and the
// scalars keep the record's order.
template <typename InT, int NP, int KS, Walk MODE, bool QLDS>
struct Stage {
  static constexpr int kK = 0;
  static constexpr int kQ = kK + TokenTile<NP, KS>::kBytes;
  static constexpr int kT = kQ + (MODE == kOutputs && QLDS ? TokenTile<NP, KS>::kBytes : 0);
  static constexpr int kP = kT + kTriBytes;
  static constexpr int kGates = kP + (MODE == kOutputs ? kTriBytes : 0);
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
  const int last = n_tokens - 1, row = min(wave * 16 + (swizzled(lane) & 15), last);  // wave w: row tile w
  o.k = static_cast<uint32_t>(row) * static_cast<uint32_t>(a.ks) * 2 + (lane >> 4) * 16;
  o.q = static_cast<uint32_t>(row) * static_cast<uint32_t>(a.qs) * 2 + (lane >> 4) * 16;
  const int col = max(0, min(col0 + (lane & 7) * 8, a.dv - 8));
#pragma unroll
  for (int i = 0; i < 2; ++i)  // 8 tokens of 64 columns
    o.v[i] = static_cast<uint32_t>(min((wave * 2 + i) * 8 + lane / 8, last)) * static_cast<uint32_t>(a.vs) * 2 + col * 2;
  return o;
}

// In four parts (PART < 0: all), which the walk issues between its products: loads
// enter the memory pipe no faster than 64 bytes a cycle, and a wave that issues them
// all at once waits for it.
template <typename InT, int KS, Walk MODE, int PART>
__device__ __forceinline__ void stage_async(char* st, const ChunkSource<InT>& s, const LaneOffsets& o, int lane,
                                            int wave) {
  using S = Stage<InT, 1, KS, MODE, true>;
  static_assert(kWaves == 4, "row tile w and values 16 w .. of wave w");
  if constexpr (PART < 0 || PART == 0) {
    const char* k = reinterpret_cast<const char*>(s.k);
#pragma unroll
    for (int i = 0; i < KS; ++i) load_to_lds(k + i * 64 + o.k, st + S::kK + (wave * KS + i) * 1024);
  }
  if constexpr (MODE == kOutputs && (PART < 0 || PART == 1)) {
    const char* q = reinterpret_cast<const char*>(s.q);
#pragma unroll
    for (int i = 0; i < KS; ++i) load_to_lds(q + i * 64 + o.q, st + S::kQ + (wave * KS + i) * 1024);
  }
  if constexpr (PART < 0 || PART >= 2) {
    const uint32_t own = lane * 16;
    constexpr int kTri = (MODE == kOutputs ? 2 * kTriBytes : kTriBytes) / 1024;
    constexpr int kAll = (kTri + kWaves - 1) / kWaves, kHalf = kAll / 2;
#pragma unroll
    for (int i = PART == 3 ? kHalf : 0; i < (PART == 2 ? kHalf : kAll); ++i) {
      const int f = wave + i * kWaves;
      if (f < kTri) load_to_lds(s.record + f * 1024 + own, st + S::kT + f * 1024);
    }
    if (PART != 2) {
      if (wave == 3) load_to_lds(s.gates + own, st + S::kGates);
      const char* v = reinterpret_cast<const char*>(s.v);
#pragma unroll
      for (int i = 0; i < 2; ++i) load_to_lds(v + o.v[i], st + S::kV + (wave * 2 + i) * 1024);
    }
  }
}

// Staging through registers, for float32 and for rows that are not whole runs.
template <typename InT, int NP, int KS, Walk MODE, bool QLDS>
__device__ __forceinline__ void stage_sync(char* st, const ChunkArgs& a, const ChunkSource<InT>& s, int col0) {
  using S = Stage<InT, NP, KS, MODE, QLDS>;
  uint16_t* sk = reinterpret_cast<uint16_t*>(st + S::kK);
  uint16_t* sq = reinterpret_cast<uint16_t*>(st + S::kQ);
  stage_rows<InT, NP, KS, kThreads>(sk, s.k, a.ks, s.n_tokens, a.dk, a.vec);
  if constexpr (MODE == kOutputs && QLDS) stage_rows<InT, NP, KS, kThreads>(sq, s.q, a.qs, s.n_tokens, a.dk, a.vec);
  constexpr int kRuns = (MODE == kOutputs ? 2 * kTriBytes : kTriBytes) / 16;
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

// Sum over the four lanes of a wave that hold the rows of one column.
__device__ __forceinline__ float column_sum(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// 0 as long as every x that went in was finite, else NaN.
__device__ __forceinline__ float finite_so_far(float so_far, float x) { return __builtin_fmaf(0.0f, x, so_far); }

// The last token up to `from` of a row at which a document starts; -1 if there is none.
__device__ __forceinline__ int64_t last_start(const uint8_t* reset, int64_t from, int lane) {
  for (int64_t t = from; t >= 0; t -= 64) {
    const uint64_t starts = __ballot(t - lane >= 0 && reset[max(t - lane, int64_t{0})] != 0);
    if (starts) return t - __builtin_ctzll(starts);
  }
  return -1;
}

// The piece's tokens again, one by one in the step form's arithmetic: a strip's outputs and,
// in H, its state after them.
//
// A chunk's products multiply 0 by whatever stands before a document's start or after a
// token, and the fold does so with the pieces before, so that a NaN or an infinity among the
// inputs reaches tokens that the recurrence keeps it from. A strip that has made a non-finite
// output therefore goes through its piece again here, and what is not finite afterwards is so
// by the recurrence. On such inputs alone it takes 2 us a token for 128 entries of k (0.8 for 48,
// 3.7 for 256; 5.5 with a load for every entry).
//
// The arguments are read anew from where the kernel was passed them, and the lane's place is
// hidden from the compiler: it would otherwise work out what it can of this ahead of the walk
// (1 x 37 x 16 heads: 18.8 us without this, 20.5 with, 19.3 so; 8 x 2048 x 12 heads: 212, 219, 215).
template <typename InT, int KS>
__device__ __forceinline__ void piece_again(int bh, int piece, int own, int lane, f32x4 (&H)[2 * KS]) {
  uint64_t passed = reinterpret_cast<uint64_t>(__builtin_amdgcn_kernarg_segment_ptr());
  asm volatile("" : "+s"(passed), "+s"(bh), "+s"(piece), "+v"(own), "+v"(lane));
  const ScanArgs& s = *reinterpret_cast<const ScanArgs*>(passed);
  const ChunkArgs& a = s.c;
  const int b = bh / a.Hv, h = bh - b * a.Hv, hk = h / a.group, g4 = (lane >> 4) * 4;
  const int64_t first = static_cast<int64_t>(piece) * s.chunks_piece * kChunk;
  const int64_t end = min(a.L, first + static_cast<int64_t>(s.chunks_piece) * kChunk);
  const bool has_v = own < a.dv;
  int64_t t = first;
  float finite = 0.0f;
#pragma unroll
  for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = state_row(m, g4, r);
      H[m][r] = 0.0f;
      if (piece > 0) {
        if (own < s.cols) H[m][r] = s.starts[((static_cast<int64_t>(bh) * s.pieces + piece) * (32 * KS) + row) * s.cols + own];
      } else if (s.h0 && row < a.dk && has_v) {
        H[m][r] = s.h0[(static_cast<int64_t>(bh) * a.dk + row) * a.dv + own];
      }
      finite = finite_so_far(finite, H[m][r]);
    }
  // Where no document starts up to here, a state that is not finite is so by the recurrence.
  if (piece > 0 && a.reset && __any(finite != 0.0f)) {
    const int64_t start = last_start(a.reset + static_cast<int64_t>(b) * a.L, first, lane);
    if (start >= 0) t = start;
  }
  const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
#pragma unroll 1
  for (; t < end; ++t) {
    const int64_t row = static_cast<int64_t>(b) * a.L + t, gate = row * a.Hv + h;
    const InT* q = static_cast<const InT*>(a.q) + row * a.qs + static_cast<int64_t>(hk) * a.dk;
    const InT* k = static_cast<const InT*>(a.k) + row * a.ks + static_cast<int64_t>(hk) * a.dk;
    const float v = has_v ? load_elem(static_cast<const InT*>(a.v), row * a.vs + static_cast<int64_t>(h) * a.dv + own) : 0.0f;
    float al = fast_exp2(A * softplus_f32(load_elem(static_cast<const InT*>(a.dt), gate) + bias) * kLog2e);
    const float beta = a.beta_scale * fast_rcp(1.0f + fast_exp2(-load_elem(static_cast<const InT*>(a.br), gate) * kLog2e));
    if (a.reset && a.reset[row]) {
      al = 0.0f;
#pragma unroll
      for (int m = 0; m < 2 * KS; ++m) H[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    f32x4 kv[2 * KS], qv[2 * KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      // the lane's eight rows 32 ks + 8 g .. of tiles 2 ks and 2 ks + 1; rows past dk are read
      // from before it and taken as 0
      const int row0 = ks * 32 + 2 * g4, last = a.dk - 1;
      float kx[8], qx[8];
      if (a.vec) {
        const int at = min(row0, last - 7);
        load8<InT, true>(k + at, 8, kx);
        load8<InT, true>(q + at, 8, qx);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          kx[i] = load_elem(k, min(row0 + i, last));
          qx[i] = load_elem(q, min(row0 + i, last));
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        kv[2 * ks + i / 4][i % 4] = row0 + i < a.dk ? kx[i] : 0.0f;
        qv[2 * ks + i / 4][i % 4] = row0 + i < a.dk ? qx[i] : 0.0f;
      }
    }
    float kh = 0.0f, qh = 0.0f, kq = 0.0f;
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        kh = __builtin_fmaf(kv[m][r], H[m][r], kh);
        qh = __builtin_fmaf(qv[m][r], H[m][r], qh);
        kq = __builtin_fmaf(kv[m][r], qv[m][r], kq);
      }
    const float u = beta * __builtin_fmaf(-al, column_sum(kh), v);
    const float o = a.scale * __builtin_fmaf(al, column_sum(qh), column_sum(kq) * u);
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) H[m][r] = __builtin_fmaf(al, H[m][r], kv[m][r] * u);
    if (t >= first && has_v && g4 == 0) {
      if (s.out_bf16)
        store_elem(static_cast<bf16_t*>(s.out), gate * a.dv + own, o);
      else
        store_elem(static_cast<float*>(s.out), gate * a.dv + own, o);
    }
  }
}

// One wave's walk over the chunks of a piece with 16 columns of the state.
//
// Bound by the chain of dependent steps of a chunk: K H0, R, T R, P U and K^T U follow
// one another, and a workgroup has a wave for every SIMD of its CU and no second one to
// fill its waits (8 x 2048 x 12 heads of 128 x 128 give 192 workgroups for 256 CUs, and the
// two staged chunks of one take 158 KB of LDS). A chunk takes about 5 us, 12000 cycles,
// 3450 of them matrix instructions: 172 us for that call, 1.8 TB/s of inputs, records and
// outputs. The 16 columns a wave are what one operand of the matrix instruction holds: more
// of them would share the operands of K, Q, T and P, but leave fewer waves than SIMDs.
// AGG: the aggregates walk (no read-out; the first 32 KS columns start from the
// identity). With two stages the next chunk is loaded while this one is worked on.
// OUT16: the output is bfloat16. Its products keep all three parts all the same, since what
// Q H0 and P U cancel of each other can be many times the output: with two parts, new values
// over old ones R times as large came out 45 x 2^-24 R off, float32 arithmetic 3 x 2^-24 R
// (and 8 x 2048 x 12 heads took 201 us, so 212).
template <typename InT, int NP, int KS, Walk MODE, bool QLDS, bool ASYNC, int STAGES, bool OUT16>
__global__ __launch_bounds__(kThreads) void delta_chunk_scan(const ScanArgs s) {
  using Tile = TokenTile<NP, KS>;
  using S = Stage<InT, NP, KS, MODE, QLDS>;
  constexpr int DKT = 2 * KS;  // row tiles of the state
  constexpr bool AGG = MODE == kAggregates, OUT = MODE == kOutputs;
  extern __shared__ __align__(16) char staged[];
  const ChunkArgs& a = s.c;
  const int lane = threadIdx.x % 64, wave = wave_index(), g4 = (lane >> 4) * 4;
  const Place place = place_of(blockIdx.x, s.col_blocks);
  if (place.item >= s.items) return;
  const int cb = place.part, piece = place.item % s.pieces, bh = place.item / s.pieces;
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
  float finite = 0.0f;  // NaN once an output is not (OUT)

  const int c0 = piece * s.chunks_piece, c1 = min(a.chunks, c0 + s.chunks_piece);
  ChunkSource<InT> src = chunk_source<InT>(s, bh, b, h, c0);
  const LaneOffsets whole = lane_offsets(a, kChunk, col0, lane, wave);
  const auto offsets = [&](int n_tokens) {
    return n_tokens == kChunk ? whole : lane_offsets(a, n_tokens, col0, lane, wave);
  };
  if constexpr (STAGES == 2) stage_async<InT, KS, MODE, -1>(staged, src, offsets(src.n_tokens), lane, wave);
  for (int c = c0; c < c1; ++c) {
    char* st = staged + (STAGES == 2 ? ((c - c0) & 1) * S::kBytes : 0);
    char* st_next = staged + (STAGES == 2 ? ((c + 1 - c0) & 1) * S::kBytes : 0);
    const bool more = c + 1 < c1;
    ChunkSource<InT> next = src;
    if (more) {
      next.q += kChunk * a.qs;
      next.k += kChunk * a.ks;
      next.v += kChunk * a.vs;
      next.record += s.record_bytes;
      next.gates += s.record_bytes;
      next.n_tokens = static_cast<int>(min(static_cast<int64_t>(kChunk), a.L - static_cast<int64_t>(c + 1) * kChunk));
    }
    const LaneOffsets next_off = offsets(next.n_tokens);  // the next chunk may be the last, with fewer tokens
    if constexpr (STAGES == 2) {
      wait_loads();
      __syncthreads();  // this stage is loaded, and the other one is no longer read
      if (more) stage_async<InT, KS, MODE, 0>(st_next, next, next_off, lane, wave);
    } else {
      __syncthreads();  // the previous chunk is no longer read
      if constexpr (ASYNC)
        stage_async<InT, KS, MODE, -1>(st, src, offsets(src.n_tokens), lane, wave);
      else
        stage_sync<InT, NP, KS, MODE, QLDS>(st, a, src, col0);
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
    // Operands of step ks + 1 are read and split while step ks is multiplied.
    f32x4 X[4] = {zero, zero, zero, zero}, Y[4] = {zero, zero, zero, zero};
    const auto load_step = [&](int ks, Frag<NP> (&kf)[4], Frag<NP> (&qf)[4]) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        kf[m] = Tile::rows(sk, m, ks, lane);
        if constexpr (OUT) {
          if constexpr (QLDS)
            qf[m] = Tile::rows(sq, m, ks, lane);
          else
            qf[m] = rows_from_global<InT>(src.q, a.qs, src.n_tokens, a.dk, a.vec, m, ks, lane);
        }
      }
    };
    Frag<3> hb = split8(H[0], H[1]);
    Frag<NP> kf[4], qf[4];
    load_step(0, kf, qf);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      Frag<3> hb_next;
      Frag<NP> kf_next[4], qf_next[4];
      if (ks + 1 < KS) {
        load_step(ks + 1, kf_next, qf_next);
        hb_next = split8(H[2 * ks + 2], H[2 * ks + 3]);
      }
      mma_n(kf, hb, X);
      if constexpr (OUT) mma_n(qf, hb, Y);
      if (ks + 1 < KS) {
        hb = hb_next;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          kf[m] = kf_next[m];
          if constexpr (OUT) qf[m] = qf_next[m];
        }
      }
    }
    if (STAGES == 2 && more) stage_async<InT, KS, MODE, 1>(st_next, next, next_off, lane, wave);
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
    if (STAGES == 2 && more) stage_async<InT, KS, MODE, 2>(st_next, next, next_off, lane, wave);
    if constexpr (OUT) {
      const Frag<3> ub[2] = {split8(U[0], U[1]), split8(U[2], U[3])};
      mma_tri(reinterpret_cast<const uint16_t*>(st + S::kP), ub, lane, Y);
    }
    if constexpr (MODE == kStates) {
      float* to = s.U + (static_cast<int64_t>(bh) * a.chunks + c) * kChunk * s.cols + own;
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (own < s.cols) to[(m * 16 + g4 + r) * s.cols] = U[m][r];
    }
    if (STAGES == 2 && more) stage_async<InT, KS, MODE, 3>(st_next, next, next_off, lane, wave);
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
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) finite = finite_so_far(finite, Y[m][r]);
      const int64_t row0 = (static_cast<int64_t>(b) * a.L + static_cast<int64_t>(c) * kChunk) * a.Hv + h;  // x dv
      if (OUT16 && (ASYNC || s.out_runs)) {  // ASYNC has whole runs everywhere
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
            if (OUT16 || s.out_bf16)
              store_elem(static_cast<bf16_t*>(s.out) + (m * 16 + r) * step, lane0, a.scale * Y[m][r]);
            else
              store_elem(static_cast<float*>(s.out) + (m * 16 + r) * step, lane0, a.scale * Y[m][r]);
          }
      }
    }
    src = next;
  }

  if (OUT && __builtin_expect(__any(finite != 0.0f), 0)) {
    __threadfence();  // what other lanes have written of the strip's outputs comes before what follows
    piece_again<InT, KS>(bh, piece, own, lane, H);
  }

  if (AGG) {
    const int width = 32 * KS + s.cols, at = strip * 16 + (lane & 15);
    if (at >= width) return;
    float* dst = s.agg + (static_cast<int64_t>(bh) * s.pieces + piece) * (32 * KS) * width + at;
#pragma unroll
    for (int m = 0; m < DKT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) dst[static_cast<int64_t>(state_row(m, g4, r)) * width] = H[m][r];
    if (s.turned && strip < DKT) {
      float* row = s.turned + ((static_cast<int64_t>(bh) * s.pieces + piece) * (32 * KS) + at) * (32 * KS);
#pragma unroll
      for (int m = 0; m < DKT; ++m) *reinterpret_cast<f32x4*>(row + state_row(m, g4, 0)) = H[m];
    }
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

template <typename InT, int NP, int KS, Walk MODE, bool QLDS, bool ASYNC, bool OUT16>
hipError_t launch_walk(const ScanArgs& s, int64_t blocks, hipStream_t stream) {
  constexpr int kBytes = Stage<InT, NP, KS, MODE, QLDS>::kBytes;
  constexpr int STAGES = ASYNC && 2 * kBytes <= kMaxLds ? 2 : 1;
  static_assert(kBytes <= kMaxLds, "a chunk's stage exceeds LDS");
  SSM_LOG("launch delta_chunk_scan<%d parts, %d rows, walk %d>: %d pieces of %d chunks, %d stages of %d bytes; "
          "grid %lld x %d threads",
          NP, 32 * KS, MODE, s.pieces, s.chunks_piece, STAGES, kBytes, static_cast<long long>(blocks), kThreads);
  hipLaunchKernelGGL((delta_chunk_scan<InT, NP, KS, MODE, QLDS, ASYNC, STAGES, OUT16>),
                     dim3(static_cast<unsigned>(blocks)), dim3(kThreads), STAGES * kBytes, stream, s);
  return hipGetLastError();
}

template <typename InT, int NP, int KS, bool ASYNC>
hipError_t launch_scan_ks(const DeltaPlan& p, const DeltaChunks& plan, ScanArgs s, hipStream_t stream) {
  // K and Q of a chunk side by side fit in LDS except for float32 past 128 entries
  constexpr bool QLDS = Stage<InT, NP, KS, kOutputs, true>::kBytes <= kMaxLds;
  const int64_t items = p.B * p.Hv * plan.pieces;
  s.items = static_cast<int>(items);
  if (plan.pieces > 1) {
    const int strips = 2 * KS + s.cols / 16;
    s.col_blocks = (strips + kWaves - 1) / kWaves;
    hipError_t e = launch_walk<InT, NP, KS, kAggregates, QLDS, ASYNC, false>(s, placed_blocks(items, s.col_blocks), stream);
    if (e != hipSuccess) return e;
    if ((e = launch_delta_fold(p, plan, s, stream)) != hipSuccess) return e;
  }
  s.col_blocks = (s.cols / 16 + kWaves - 1) / kWaves;
  const int64_t blocks = placed_blocks(items, s.col_blocks);
  if (s.states) return launch_walk<InT, NP, KS, kStates, QLDS, ASYNC, false>(s, blocks, stream);
  if (NP == 1 && s.out_bf16) return launch_walk<InT, NP, KS, kOutputs, QLDS, ASYNC, NP == 1>(s, blocks, stream);
  return launch_walk<InT, NP, KS, kOutputs, QLDS, ASYNC, false>(s, blocks, stream);
}

template <typename InT, int NP, bool ASYNC>
hipError_t launch_all(const DeltaPlan& p, const DeltaChunks& plan, const ScanArgs& s, hipStream_t stream) {
  switch (padded_ks(p.dk)) {
    case 1: return launch_scan_ks<InT, NP, 1, ASYNC>(p, plan, s, stream);
    case 2: return launch_scan_ks<InT, NP, 2, ASYNC>(p, plan, s, stream);
    case 3: return launch_scan_ks<InT, NP, 3, ASYNC>(p, plan, s, stream);
    case 4: return launch_scan_ks<InT, NP, 4, ASYNC>(p, plan, s, stream);
    case 6: return launch_scan_ks<InT, NP, 6, ASYNC>(p, plan, s, stream);
    default: return launch_scan_ks<InT, NP, 8, ASYNC>(p, plan, s, stream);
  }
}

}  // namespace
}  // namespace ssm
