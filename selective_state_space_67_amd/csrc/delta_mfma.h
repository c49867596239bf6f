// Matrix-core building blocks of the chunked gated delta rule (gfx950).
//
// Every product is v_mfma_f32_16x16x32_bf16 with float32 sums. A float32
// operand goes in as three bfloat16 parts that add up to it exactly (8 bits of
// the significand each); a bfloat16 input is its own single part. Products of
// parts below 2^-26 of the whole are left out, so an operand costs 3 products
// against an input part and 6 against another split operand, and results carry
// float32's precision. (The float32 matrix instructions run at 1/16 of the
// bfloat16 rate.)
//
// Lane layouts (lane l, g = l / 16): A holds row l % 16 and 8 entries of the
// summed index, B column l % 16 and the same 8; D holds column l % 16 and rows
// 4 g .. 4 g + 3. The order of the summed index is free as long as A and B agree,
// and it is chosen so that two D tiles are a B operand as they stand: slots 0..3
// of lane group g are rows 4 g .. of the first, slots 4..7 those of the second.
// A chain of products on one 16-column strip therefore never leaves the
// registers. Rows of a D tile stand for
//   tokens:  row 4 g + r of tile m is token 16 m + 4 g + r;
//   entries of k and q (rows of the state): row 4 g + r of tile 2 s + t is entry
//            32 s + 8 g + 4 t + r, so that a lane's 8 slots are 8 neighbours and a
//            token's row is staged in 16-byte runs.
#pragma once

#include "device_math.h"

namespace ssm {

constexpr int kChunk = 64;  // tokens per chunk

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The wave's place in its workgroup as a scalar. Matrix instructions run whatever
// the lane mask says, so a product under a condition on the wave needs a branch the
// compiler knows to be uniform; a mask would not keep it from running.
__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x / 64); }

// Workgroups go round the 8 dies in turn, each with an L2 of its own: the parts of an
// item, which read the same tokens and records, are 8 apart and share one. (With the parts
// next to each other the walk of 8 x 2048 x 12 heads fetched 426 MB, so 237; its reverse 462
// and 255.)
constexpr int kDies = 8;
struct Place {
  int item, part;  // item: may be past the last one
};
__device__ __forceinline__ Place place_of(int block, int parts) {
  const int round = block / (kDies * parts), in = block - round * kDies * parts;
  return {round * kDies + in % kDies, in / kDies};
}
inline int64_t placed_blocks(int64_t items, int parts) { return (items + kDies - 1) / kDies * kDies * parts; }

// An operand of one product: NP parts of 8 entries.
template <int NP>
struct Frag {
  u32x4 p[NP];
};

// Two floats rounded to bfloat16 (nearest even), lo in the low half: one conversion.
__device__ __forceinline__ uint32_t bf16_words(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// Two floats in three parts, each the rest rounded to bfloat16: the rest after two
// roundings to 8 bits has at most 8 left, so the three add up exactly, and a part is
// at most 2^-9 of the one before it.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&w)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    w[i] = bf16_words(a, b);
    a -= __uint_as_float(w[i] << 16);
    b -= __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Two D tiles (or any two runs of four) as a split operand.
__device__ __forceinline__ Frag<3> split8(f32x4 a, f32x4 b) {
  Frag<3> f;
  uint32_t w[3];
  split_pair(a.x, a.y, w);
#pragma unroll
  for (int i = 0; i < 3; ++i) f.p[i].x = w[i];
  split_pair(a.z, a.w, w);
#pragma unroll
  for (int i = 0; i < 3; ++i) f.p[i].y = w[i];
  split_pair(b.x, b.y, w);
#pragma unroll
  for (int i = 0; i < 3; ++i) f.p[i].z = w[i];
  split_pair(b.z, b.w, w);
#pragma unroll
  for (int i = 0; i < 3; ++i) f.p[i].w = w[i];
  return f;
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}

// Four entries a lane from a 4 x 16 block of 16-bit entries that a group of 16 lanes
// names in runs of four (lane i: row i / 4, run i % 4): lane i receives column i.
__device__ __forceinline__ u32x2 read_transposed(const uint16_t* p) {
  using lds_t = __attribute__((address_space(3))) s16x4*;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(p)));
}

// c += a b, smallest parts first.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Frag<NA>& a, const Frag<NB>& b, f32x4 c) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) c = mfma(a.p[i], b.p[s - i], c);
  return c;
}

// Entry of k (row of the state) that row 4 g + r of tile m stands for; g4 = 4 g.
__device__ __forceinline__ int state_row(int m, int g4, int r) { return (m >> 1) * 32 + g4 * 2 + (m & 1) * 4 + r; }

// c[n] += a[n] b for N independent sums, in turns: a sum's next product waits for
// its last one, the others' do not.
template <int N, int NA, int NB>
__device__ __forceinline__ void mma_n(const Frag<NA> (&a)[N], const Frag<NB>& b, f32x4 (&c)[N]) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB)
#pragma unroll
        for (int n = 0; n < N; ++n) c[n] = mfma(a[n].p[i], b.p[s - i], c[n]);
}

// c[n] += a b[n] for two independent sums, in turns.
template <int NA, int NB>
__device__ __forceinline__ void mma_b(const Frag<NA>& a, const Frag<NB> (&b)[2], f32x4* c) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) {
        c[0] = mfma(a.p[i], b[0].p[s - i], c[0]);
        c[1] = mfma(a.p[i], b[1].p[s - i], c[1]);
      }
}
// c += a b and d += e f, in turns.
template <int NA, int NB>
__device__ __forceinline__ void mma_pair(const Frag<NA>& a, const Frag<NB>& b, f32x4& c, const Frag<NA>& e,
                                         const Frag<NB>& f, f32x4& d) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) {
        c = mfma(a.p[i], b.p[s - i], c);
        d = mfma(e.p[i], f.p[s - i], d);
      }
}

// Rows of tokens staged in LDS as A operands: parts x (64 / 16 tiles of rows) x
// (KS tiles of 32 entries) x 64 lanes x 8 entries. Within a tile lane l's run lies at
// swizzled(l): the four runs of one token's 64 bytes then fall on different banks, both
// when threads that loaded neighbouring bytes store them and when a transposing read
// takes them. 16-byte reads of whole operands stay free of conflicts only with these
// turns (0, 3, 2, 1 blocks of four tokens): with 0, 1, 2, 3 the conflict cycles of the
// preparing kernel rose 13-fold (1.2e5 to 1.6e6, 8 x 2048 x 12 heads); with none those
// of the gradients' kernel were 3.7e7, now 1.2e7, and its time 420 us, now 360.
__device__ __forceinline__ int swizzled(int lane) { return lane ^ ((lane >> 4) * 12 & 12); }

template <int NP, int KS>
struct TokenTile {
  static constexpr int kFrags = 4 * KS;
  static constexpr int kPart = kFrags * 64 * 8;  // entries of one part
  static constexpr int kBytes = NP * kPart * 2;

  // Offset, in entries, of the run of eight entries 8 * oct .. of a token.
  __device__ __forceinline__ static int at(int token, int oct) {
    return (((token >> 4) * KS + (oct >> 2)) * 64 + swizzled((oct & 3) * 16 + (token & 15))) * 8;
  }
  // A operand with the tokens of tile mi as rows, summed over entries 32 ks ..
  __device__ __forceinline__ static Frag<NP> rows(const uint16_t* s, int mi, int ks, int lane) {
    Frag<NP> f;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      f.p[i] = *reinterpret_cast<const u32x4*>(s + i * kPart + ((mi * KS + ks) * 64 + swizzled(lane)) * 8);
    return f;
  }
  // A operand with the entries of state tile m0 as rows, summed over tokens 32 ts ..:
  // transposing reads, where each group of 16 lanes names 4 tokens x 4 runs of four
  // entries (lane i: token i / 4, run i % 4) and lane i receives entry i of the 4 tokens.
  __device__ __forceinline__ static Frag<NP> columns(const uint16_t* s, int m0, int ts, int lane) {
    const int token = ts * 32 + (lane >> 4) * 4 + ((lane & 15) >> 2), oct = (m0 >> 1) * 4 + (lane & 3);
    Frag<NP> f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint16_t* p = s + i * kPart + (m0 & 1) * 4;
      const u32x2 lo = read_transposed(p + at(token, oct)), hi = read_transposed(p + at(token + 16, oct));
      f.p[i] = u32x4{lo.x, lo.y, hi.x, hi.y};
    }
    return f;
  }
};

// Eight consecutive entries of a token from global memory; entries at or past
// `left` are 0. VEC: whole and aligned.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int left, float (&x)[8]) {
  if constexpr (VEC) {
    constexpr int per = 16 / static_cast<int>(sizeof(T));
#pragma unroll
    for (int i = 0; i < 8; i += per) {
      const typename Run<T, per>::raw w = Run<T, per>::load(p + i);
#pragma unroll
      for (int j = 0; j < per; ++j) x[i + j] = Run<T, per>::at(w, j);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < left ? load_elem(p, i) : 0.0f;
  }
}

// Stage tokens 0 .. n_tokens - 1 (0 beyond) and entries d0 .. d0 + 32 KS - 1 (0 at or
// past d) of a token-strided tensor. All threads of the workgroup call it.
template <typename T, int NP, int KS, bool VEC, int THREADS>
__device__ __forceinline__ void stage_tokens(uint16_t* s, const T* src, int64_t stride, int n_tokens, int d0, int d) {
  using Tile = TokenTile<NP, KS>;
  constexpr int kOct = KS * 4;  // runs of 8 entries per token
#pragma unroll
  for (int i = threadIdx.x; i < 64 * kOct; i += THREADS) {
    // a wave takes 16 tokens x 4 runs: 64 or 128 bytes of each token's row
    const int token = (i & 15) | ((i / (16 * kOct)) << 4), oct = (i >> 4) % kOct;
    const int left = d - d0 - oct * 8;
    const T* p = src + token * stride + d0 + oct * 8;
    uint16_t* to = s + Tile::at(token, oct);
    if constexpr (NP == 1) {
      u32x4 w = {0, 0, 0, 0};
      if (token < n_tokens && left > 0) {
        if constexpr (VEC) {
          w = *reinterpret_cast<const u32x4*>(p);
        } else {
          uint32_t e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = j < left ? p[j].bits : 0u;
          w = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
        }
      }
      *reinterpret_cast<u32x4*>(to) = w;
    } else {
      float x[8] = {};
      if (token < n_tokens && left > 0) load8<T, VEC>(p, left, x);
      const Frag<3> f = split8(f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]});
#pragma unroll
      for (int k = 0; k < 3; ++k) *reinterpret_cast<u32x4*>(to + k * Tile::kPart) = f.p[k];
    }
  }
}

// All 32 KS entries, whole runs or not as `vec` says.
template <typename T, int NP, int KS, int THREADS>
__device__ __forceinline__ void stage_rows(uint16_t* s, const T* src, int64_t stride, int n_tokens, int d, bool vec) {
  if (vec)
    stage_tokens<T, NP, KS, true, THREADS>(s, src, stride, n_tokens, 0, d);
  else
    stage_tokens<T, NP, KS, false, THREADS>(s, src, stride, n_tokens, 0, d);
}

// A operand like TokenTile::rows, straight from global memory and split on the
// way (where the tile does not fit in LDS). `src`: the chunk's first token.
template <typename T>
__device__ __forceinline__ Frag<3> rows_from_global(const T* src, int64_t stride, int n_tokens, int d, bool vec, int mi,
                                                    int ks, int lane) {
  const int token = mi * 16 + (lane & 15), at = ks * 32 + (lane >> 4) * 8;
  float x[8] = {};
  if (token < n_tokens && at < d) {
    if (vec)
      load8<T, true>(src + token * stride + at, d - at, x);
    else
      load8<T, false>(src + token * stride + at, d - at, x);
  }
  return split8(f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]});
}

// 16 bytes a lane from global memory straight into LDS: lane l's go to dst + 16 l
// (dst the same in the whole wave). Done when the wave's loads are waited for.
__device__ __forceinline__ void load_to_lds(const void* src, void* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// Stage 64 tokens like stage_tokens, straight into LDS: bfloat16 rows of 32 KS whole
// entries, by four waves (wave w: row tile w); tokens past the end repeat the last.
template <int KS>
__device__ __forceinline__ void stage_tokens_async(uint16_t* s, const bf16_t* src, int64_t stride, int n_tokens,
                                                   int lane, int wave) {
  const int row = min(wave * 16 + (swizzled(lane) & 15), n_tokens - 1);
  const char* p = reinterpret_cast<const char*>(src + row * stride) + (lane >> 4) * 16;
#pragma unroll
  for (int i = 0; i < KS; ++i) load_to_lds(p + i * 64, s + (wave * KS + i) * 512);
}

// Everything this wave has loaded has arrived.
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }  // vmcnt(0)

// A chunk's triangular 64 x 64 matrix as split A operands in global memory: for
// row tile mi the summed tiles ks <= mi / 2 (mi, ks) -> 6 operands, or for its
// transpose ks >= mi / 2; three parts x 6 operands x 64 lanes x 8 entries.
constexpr int kTriFrags = 6;
constexpr int kTriEntries = kTriFrags * 3 * 64 * 8;
constexpr int kTriBytes = kTriEntries * 2;
__host__ __device__ constexpr int tri_index(int mi, int ks) { return mi < 2 ? mi : 2 + (mi - 2) * 2 + ks; }
// transposed: row tiles 0 and 1 sum over both halves, 2 and 3 over the second
__host__ __device__ constexpr int tri_t_index(int mi, int ks) { return mi < 2 ? mi * 2 + ks : mi + 2; }

// Operand `index`; its parts lie one after another.
__device__ __forceinline__ Frag<3> load_tri(const uint16_t* m, int index, int lane) {
  Frag<3> f;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    f.p[i] = *reinterpret_cast<const u32x4*>(m + ((i * kTriFrags + index) * 64 + lane) * 8);
  return f;
}
__device__ __forceinline__ void store_tri(uint16_t* m, int index, int lane, const Frag<3>& f) {
#pragma unroll
  for (int i = 0; i < 3; ++i) *reinterpret_cast<u32x4*>(m + ((i * kTriFrags + index) * 64 + lane) * 8) = f.p[i];
}

// c[m] += M[m][.] b for the four row tiles of a staged triangle M (rows m sum over
// the halves ks <= m / 2): six independent sums in turns.
__device__ __forceinline__ void mma_tri(const uint16_t* m, const Frag<3> (&b)[2], int lane, f32x4 (&c)[4]) {
  Frag<3> a[6];
#pragma unroll
  for (int i = 0; i < 6; ++i) a[i] = load_tri(m, i, lane);
  f32x4 d[2] = {};
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i <= s; ++i) {
      c[0] = mfma(a[0].p[i], b[0].p[s - i], c[0]);
      c[1] = mfma(a[1].p[i], b[0].p[s - i], c[1]);
      c[2] = mfma(a[2].p[i], b[0].p[s - i], c[2]);
      c[3] = mfma(a[4].p[i], b[0].p[s - i], c[3]);
      d[0] = mfma(a[3].p[i], b[1].p[s - i], d[0]);
      d[1] = mfma(a[5].p[i], b[1].p[s - i], d[1]);
    }
  c[2] += d[0];
  c[3] += d[1];
}

// The same for a transposed triangle (rows m sum over the halves ks >= m / 2).
template <int NB>
__device__ __forceinline__ void mma_tri_t(const uint16_t* m, const Frag<NB> (&b)[2], int lane, f32x4 (&c)[4]) {
  Frag<3> a[6];
#pragma unroll
  for (int i = 0; i < 6; ++i) a[i] = load_tri(m, i, lane);
  f32x4 d[2] = {};
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i <= s; ++i) {
      if (s - i >= NB) continue;
      c[0] = mfma(a[0].p[i], b[0].p[s - i], c[0]);
      c[1] = mfma(a[2].p[i], b[0].p[s - i], c[1]);
      c[2] = mfma(a[4].p[i], b[1].p[s - i], c[2]);
      c[3] = mfma(a[5].p[i], b[1].p[s - i], c[3]);
      d[0] = mfma(a[1].p[i], b[1].p[s - i], d[0]);
      d[1] = mfma(a[3].p[i], b[1].p[s - i], d[1]);
    }
  c[0] += d[0];
  c[1] += d[1];
}

// Per-chunk scalars, eight rows of 64 tokens:
//   e0 = exp(sum of log decays from the chunk's start through the token), 0 after a reset;
//        the last token's, aC, is the whole chunk's decay
//   eC = exp(sum after the token to the chunk's end), 0 before a reset
//   beta; the derivative of softplus at the token's step size
// and for the backward the sums themselves (in log2 units, as two floats), the number
// of documents started in the chunk up to the token, and the step size.
constexpr int kE0 = 0, kAC = 63, kEC = 64, kBeta = 128, kSlope = 192;
constexpr int kSumHi = 256, kSumLo = 320, kSeg = 384, kDelta = 448;
constexpr int kGateFloats = 256;     // what the walks read
constexpr int kGateFloatsBwd = 512;

}  // namespace ssm
