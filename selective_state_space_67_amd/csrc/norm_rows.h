// Rows for the norms around a block (gated_norm.hip, block_norm.hip): a team of
// lanes holds a row in registers, NV runs of V elements a lane, run j of lane i at
// element (j team + i) V. A team is TR = 8 to 64 lanes of a wave, or (TR = 0) a
// whole workgroup of as many waves as the row needs. The only exchange is the sum
// over the row, by DPP within a wave and through LDS between waves.
//
// V = 8 (16 bytes of bfloat16) needs sizes and addresses in multiples of a run;
// V = 1 takes everything else. A team goes through its rows in strides, and the
// next row is loaded (as it lies in memory, half the registers of bfloat16) while
// one is worked on.
#pragma once

#include <algorithm>

#include "device_math.h"
#include "kernels_block.h"
#include "lane_sums.h"

namespace ssm {

// V elements as they lie in memory, and as floats.
template <int V, typename T>
struct Raw {
  static constexpr int kWords = V == 1 ? 1 : V * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V == 1) {
      if constexpr (sizeof(T) == 2)
        w[0] = reinterpret_cast<const uint16_t*>(p)[0];
      else
        w[0] = reinterpret_cast<const uint32_t*>(p)[0];
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 r = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
        w[i] = r.x;
        w[i + 1] = r.y;
        w[i + 2] = r.z;
        w[i + 3] = r.w;
      }
    }
  }
  // from a buffer: zeros past its end
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, uint32_t offset) {
    if constexpr (V == 1) {
      if constexpr (sizeof(T) == 2)
        w[0] = __builtin_amdgcn_raw_buffer_load_b16(b, offset, 0, 0);
      else
        w[0] = __builtin_amdgcn_raw_buffer_load_b32(b, offset, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const auto r = __builtin_amdgcn_raw_buffer_load_b128(b, offset + 4 * i, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[i + k] = r[k];
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    if constexpr (V == 1) return __uint_as_float(w[0] << 16);
    return __uint_as_float((i & 1) ? (w[i / 2] & 0xFFFF0000u) : (w[i / 2] << 16));
  }
};

// Two floats as bfloat16, nearest even, by the hardware's conversion (a NaN stays one).
__device__ __forceinline__ uint32_t bf16_two(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// A row of `bytes` bytes as a buffer: what is read past its end is 0, what is written there is dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const void* row, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(row), 0, bytes, 0x00020000);
}

typedef uint32_t words4 __attribute__((ext_vector_type(4)));

// V results as the words that bfloat16 or float32 takes.
template <int V>
__device__ __forceinline__ words4 bf16_words4(const float (&x)[V]) {
  return words4{bf16_two(x[0], x[1]), bf16_two(x[2], x[3]), bf16_two(x[4], x[5]), bf16_two(x[6], x[7])};
}
__device__ __forceinline__ words4 float_words4(const float* x) {
  return words4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
}

template <int V>
__device__ __forceinline__ void store_run(char* p, bool bf16, const float (&x)[V]) {
  if constexpr (V == 1) {
    if (bf16)
      *reinterpret_cast<uint16_t*>(p) = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x[0]));
    else
      *reinterpret_cast<float*>(p) = x[0];
  } else if (bf16) {
    *reinterpret_cast<words4*>(p) = bf16_words4(x);
  } else {
    *reinterpret_cast<words4*>(p) = float_words4(x);
    *reinterpret_cast<words4*>(p + 16) = float_words4(x + 4);
  }
}
template <int V>
__device__ __forceinline__ void store_run(__amdgpu_buffer_rsrc_t b, uint32_t offset, bool bf16, const float (&x)[V]) {
  if constexpr (V == 1) {
    if (bf16)
      __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, static_cast<__bf16>(x[0])), b, offset, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[0]), b, offset, 0, 0);
  } else if (bf16) {
    __builtin_amdgcn_raw_buffer_store_b128(bf16_words4(x), b, offset, 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b128(float_words4(x), b, offset, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b128(float_words4(x + 4), b, offset + 16, 0, 0);
  }
}

// Where a lane's runs lie in a row of `size` elements.
template <int V, int TR, int NV>
struct Columns {
  int lane, team, size;
  __device__ __forceinline__ Columns(int size)
      : lane(TR ? threadIdx.x % TR : threadIdx.x), team(TR ? TR : blockDim.x), size(size) {}
  __device__ __forceinline__ int at(int j) const { return (j * team + lane) * V; }
  __device__ __forceinline__ bool on(int j) const { return at(j) < size; }

  // A row as it lies in memory; runs past its end are zeros. A workgroup's row goes through a
  // buffer, so that its runs need neither addresses nor masks.
  template <typename T>
  __device__ __forceinline__ void load(const void* base, int64_t row, Raw<V, T> (&x)[NV]) const {
    const T* p = static_cast<const T*>(base) + row;
    if constexpr (TR == 0) {
      const auto b = row_buffer(p, size * static_cast<int>(sizeof(T)));
#pragma unroll
      for (int j = 0; j < NV; ++j) x[j].load(b, static_cast<uint32_t>(at(j)) * sizeof(T));
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        x[j] = Raw<V, T>{};
        if (on(j)) x[j].load(p + at(j));
      }
    }
  }
  // a weight row: 1 where there is none
  __device__ __forceinline__ void weights(const float* w, float (&x)[NV][V]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) x[j][i] = 1.0f;
    if (!w) return;
    Raw<V, float> r[NV];
    load(w, 0, r);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) x[j][i] = r[j].at(i);
  }
  __device__ __forceinline__ void store(void* base, int64_t row, bool bf16, const float (&x)[NV][V]) const {
    const int bytes = bf16 ? 2 : 4;
    char* p = static_cast<char*>(base) + row * bytes;
    if constexpr (TR == 0) {
      const auto b = row_buffer(p, size * bytes);
#pragma unroll
      for (int j = 0; j < NV; ++j) store_run<V>(b, static_cast<uint32_t>(at(j)) * bytes, bf16, x[j]);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on(j)) store_run<V>(p + at(j) * bytes, bf16, x[j]);
    }
  }
};

// Sum over the row's team, in all of its lanes. The sums of a team of several waves take
// turns in two halves of LDS, so that one barrier serves each.
template <int TR>
class TeamSum {
 public:
  __device__ __forceinline__ float operator()(float x, float (&lds)[2][16]) {
    if constexpr (TR != 0) {
      return lanes_sum<TR>(x);
    } else {
      x = lanes_sum<64>(x);
      if (threadIdx.x % 64 == 0) lds[half_][threadIdx.x / 64] = x;
      __syncthreads();
      const int i = threadIdx.x % 16;
      x = i < static_cast<int>(blockDim.x / 64) ? lds[half_][i] : 0.0f;
      half_ ^= 1;
      return lanes_sum<16>(x);
    }
  }

 private:
  int half_ = 0;
};

template <int NV, int V>
__device__ __forceinline__ float dot(const float (&a)[NV][V], const float (&b)[NV][V]) {
  float t = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) t = __builtin_fmaf(a[j][i], b[j][i], t);
  return t;
}

// The rows that a team works on, in strides: those of one group (rows that share their
// weights and the sums of their gradients), cut into parts, a workgroup each.
struct RowWalk {
  int64_t row, end, step;
  template <int TR>
  __device__ __forceinline__ static RowWalk of(const RowGroups& g) {
    const int teams = TR ? blockDim.x / (TR ? TR : 1) : 1, part = blockIdx.x % g.parts;
    const int64_t first = static_cast<int64_t>(part) * teams + (TR ? threadIdx.x / (TR ? TR : 1) : 0);
    return {first, g.rows, static_cast<int64_t>(g.parts) * teams};
  }
  __device__ __forceinline__ static int group(const RowGroups& g) { return blockIdx.x / g.parts; }
};

// A workgroup's sums over its rows: its teams' are added up in LDS (`lds` holds `size` floats
// for each) in their order.
template <int V, int TR, int NV>
__device__ __forceinline__ void store_sums(const Columns<V, TR, NV>& c, const float (&x)[NV][V], float* lds, float* to) {
  if constexpr (TR == 0) {
    c.store(to, 0, false, x);
  } else {
    __syncthreads();
    float* mine = lds + (threadIdx.x / TR) * c.size;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (c.on(j)) {
#pragma unroll
        for (int i = 0; i < V; ++i) mine[c.at(j) + i] = x[j][i];
      }
    __syncthreads();
    for (int e = threadIdx.x; e < c.size; e += blockDim.x) {
      float t = 0.0f;
      for (int k = 0; k < static_cast<int>(blockDim.x / TR); ++k) t += lds[k * c.size + e];
      to[e] = t;
    }
  }
}

// Team shapes for a row of `size` elements, and the threads of a workgroup: 256 of several
// teams (64 where that would leave CUs idle: `rows` rows in all), or as many as a row needs.
// F::run<V, TR, NV, most threads>(threads, ...); F::kMany: it holds many rows of sums.
template <typename F, typename... X>
hipError_t pick_team(bool runs, int size, int64_t rows, X&&... x) {
  auto several = [&](int team) { return rows >= 256 * (256 / team) ? 256 : 64; };
  auto whole = [&](int each) { return (size + 64 * each - 1) / (64 * each) * 64; };
  if (runs) {
    if (size <= 64) return F::template run<8, 8, 1, 256>(several(8), std::forward<X>(x)...);
    if (size <= 128) return F::template run<8, 16, 1, 256>(several(16), std::forward<X>(x)...);
    if (size <= 256) return F::template run<8, 32, 1, 256>(several(32), std::forward<X>(x)...);
    if (size <= 512) return F::template run<8, 64, 1, 256>(several(64), std::forward<X>(x)...);
    if (size <= 4096) return F::template run<8, 0, 1, 512>(whole(8), std::forward<X>(x)...);
    if (size <= 8192) return F::template run<8, 0, 1, 1024>(whole(8), std::forward<X>(x)...);
    return F::template run<8, 0, 2, 1024>(whole(16), std::forward<X>(x)...);
  }
  if (size <= 32) return F::template run<1, 8, 4, 256>(several(8), std::forward<X>(x)...);
  if (size <= 64) return F::template run<1, 16, 4, 256>(several(16), std::forward<X>(x)...);
  if (size <= 128) return F::template run<1, 32, 4, 256>(several(32), std::forward<X>(x)...);
  if (size <= 256) return F::template run<1, 64, 4, 256>(several(64), std::forward<X>(x)...);
  if (size <= 512) return F::template run<1, 64, 8, 256>(several(64), std::forward<X>(x)...);
  if (size <= 4096) return F::template run<1, 0, 8, 512>(whole(8), std::forward<X>(x)...);
  // Twice as many entries a lane in half as many waves, where a lane has many registers' worth of rows
  // and sums: backward of the block norm, 5118 rows of 4097, 242 -> 154 us (its forward 50 -> 65, the
  // gated norm's backward 83 -> 109).
  if constexpr (F::kMany) {
    if (size <= 8192) return F::template run<1, 0, 16, 512>(whole(16), std::forward<X>(x)...);
  } else {
    if (size <= 8192) return F::template run<1, 0, 8, 1024>(whole(8), std::forward<X>(x)...);
  }
  return F::template run<1, 0, 16, 1024>(whole(16), std::forward<X>(x)...);
}

// What a lane's registers hold besides a row: the next one's elements unless its runs are long or
// (a kernel with many rows of sums) its workgroup so large that it has no more than 128 registers,
// and the weights unless its runs are long.
template <int V, int NV, int MOST, bool MANY>
struct Holds {
  static constexpr bool kAhead = V * NV <= 8 && (!MANY || MOST <= 512), kWeights = V * NV <= 8;
};

// Threads that go through the rows: 2048 a CU.
constexpr int64_t kWantThreads = int64_t{1} << 19;

// Parts of a group of rows, for a launch of that many threads; `teams` rows at once in a workgroup.
inline int row_parts(const RowGroups& g, int threads, int teams) {
  const int64_t most = (g.rows + teams - 1) / teams;
  return static_cast<int>(std::min(most, std::max<int64_t>(1, kWantThreads / threads / g.groups)));
}

// Workgroups of a backward, each of which leaves a row of sums for the weights: the least whole
// number for every CU that gives it `per_cu` threads (a part more on some CUs makes the others
// wait: 4096 rows of 5120 of the block norm 85 us with 256 workgroups, 115 with 307). Few rows:
// one for 8192 entries or 8 rows (a row after another takes a team 0.6 us and more).
inline int64_t row_sum_blocks(int64_t groups, int64_t rows, int size, int64_t per_cu) {
  const int64_t threads = size <= 512 ? 256 : (size + 511) / 512 * 64;
  const int64_t most = std::max<int64_t>(1, 256 * ((per_cu + threads - 1) / threads) / groups);
  const int64_t want = std::min(std::max((rows * size + 8191) / 8192, rows / 8), most);
  return groups * std::max<int64_t>(1, std::min(want, rows));
}

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace ssm
