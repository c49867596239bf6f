// Rows for the norms around a block (gated_norm.hip, block_norm.hip): a team of
// TR lanes holds a row in registers, NV runs of V elements a lane, run j of lane
// i at element (j TR + i) V. The only exchange is the sum over the row, by DPP
// within a wave and through LDS between the waves of a larger team.
//
// V = 8 (16 bytes of bfloat16) needs sizes and addresses in multiples of a run;
// V = 1 takes everything else.
#pragma once

#include <algorithm>

#include "device_math.h"
#include "kernels_block.h"
#include "lane_sums.h"

namespace ssm {

// V elements as floats from / to memory of type T.
template <int V, typename T>
__device__ __forceinline__ void load_run(const T* p, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = load_elem(p, 0);
  } else if constexpr (sizeof(T) == 2) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t q = word(r, i >> 1);
      x[i] = __uint_as_float((i & 1) ? (q & 0xFFFF0000u) : (q << 16));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 r = *reinterpret_cast<const float4*>(p + i);
      x[i] = r.x;
      x[i + 1] = r.y;
      x[i + 2] = r.z;
      x[i + 3] = r.w;
    }
  }
}

// Two floats as bfloat16, nearest even, by the hardware's conversion (a NaN stays one).
__device__ __forceinline__ uint32_t bf16_two(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

template <int V>
__device__ __forceinline__ void store_run(void* base, int64_t at, bool bf16, const float (&x)[V]) {
  if (bf16) {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    if constexpr (V == 1)
      *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x[0]));
    else
      *reinterpret_cast<uint4*>(p) = make_uint4(bf16_two(x[0], x[1]), bf16_two(x[2], x[3]), bf16_two(x[4], x[5]),
                                                bf16_two(x[6], x[7]));
  } else {
    float* p = static_cast<float*>(base) + at;
    if constexpr (V == 1) {
      *p = x[0];
    } else {
      *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
}

// Where a lane's runs lie in a row of `size` elements.
template <int V, int TR, int NV>
struct Columns {
  int lane, size;
  __device__ __forceinline__ Columns(int size) : lane(threadIdx.x % TR), size(size) {}
  __device__ __forceinline__ int at(int j) const { return (j * TR + lane) * V; }
  __device__ __forceinline__ bool on(int j) const { return at(j) < size; }

  template <typename T>
  __device__ __forceinline__ void load(const T* row, float (&x)[NV][V]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (on(j)) {
        load_run<V>(row + at(j), x[j]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[j][i] = 0.0f;
      }
    }
  }
  // a weight row: 1 where there is none
  __device__ __forceinline__ void weights(const float* w, float (&x)[NV][V]) const {
    if (w) {
      load(w, x);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) x[j][i] = 1.0f;
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t row, bool bf16, const float (&x)[NV][V]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (on(j)) store_run<V>(base, row + at(j), bf16, x[j]);
  }
};

// Sum over the row's team, in all of its lanes. A team of several waves is the whole
// workgroup; its sums take turns in two halves of LDS, so that one barrier serves each.
template <int TR>
class TeamSum {
 public:
  static constexpr int kWaves = TR > 64 ? TR / 64 : 1;
  __device__ __forceinline__ float operator()(float x, float (&lds)[2][kWaves]) {
    if constexpr (TR <= 64) {
      return lanes_sum<TR>(x);
    } else {
      x = lanes_sum<64>(x);
      if (threadIdx.x % 64 == 0) lds[half_][threadIdx.x / 64] = x;
      __syncthreads();
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) t += lds[half_][i];
      half_ ^= 1;
      return t;
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
    const int teams = blockDim.x / TR, part = blockIdx.x % g.parts;
    const int64_t first = static_cast<int64_t>(part) * teams + threadIdx.x / TR;
    return {first, g.rows, static_cast<int64_t>(g.parts) * teams};
  }
  __device__ __forceinline__ static int group(const RowGroups& g) { return blockIdx.x / g.parts; }
};

// A workgroup's sums over its teams' rows: added up in LDS in the teams' order, one row of
// `count` x size sums a workgroup. `lds` holds size floats for each team.
template <int V, int TR, int NV>
__device__ __forceinline__ void store_sums(const Columns<V, TR, NV>& c, const float (&x)[NV][V], float* lds, float* to) {
  const int teams = blockDim.x / TR;
  if (teams == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (c.on(j)) {
#pragma unroll
        for (int i = 0; i < V; ++i) to[c.at(j) + i] = x[j][i];
      }
    return;
  }
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
    for (int k = 0; k < teams; ++k) t += lds[k * c.size + e];
    to[e] = t;
  }
}

// Team shapes for a row of `size` elements: F::run<V, TR, NV>(...). Up to 16 elements a lane.
template <typename F, typename... X>
hipError_t pick_team(bool runs, int size, X&&... x) {
  if (runs) {
    if (size <= 512) return F::template run<8, 64, 1>(std::forward<X>(x)...);
    if (size <= 1024) return F::template run<8, 64, 2>(std::forward<X>(x)...);
    if (size <= 2048) return F::template run<8, 256, 1>(std::forward<X>(x)...);
    if (size <= 4096) return F::template run<8, 256, 2>(std::forward<X>(x)...);
    if (size <= 8192) return F::template run<8, 512, 2>(std::forward<X>(x)...);
    return F::template run<8, 1024, 2>(std::forward<X>(x)...);
  }
  if (size <= 256) return F::template run<1, 64, 4>(std::forward<X>(x)...);
  if (size <= 1024) return F::template run<1, 64, 16>(std::forward<X>(x)...);
  if (size <= 4096) return F::template run<1, 256, 16>(std::forward<X>(x)...);
  return F::template run<1, 1024, 16>(std::forward<X>(x)...);
}

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// Threads of a workgroup: a team, or 256 of several teams (64 where that leaves CUs idle).
template <int TR>
int workgroup_threads(int64_t rows) {
  if (TR >= 256) return TR;
  const int64_t teams = 256 / TR;
  return rows >= teams * 256 || TR > 64 ? 256 : std::max(TR, 64);
}

}  // namespace ssm
