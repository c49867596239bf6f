// Sums over the workgroups' rows of partial sums (weights' gradients of the norms
// around a block): 16 columns a workgroup, 16 threads a column, each adding every
// 16th row in order with eight of them under way, then the 16 sums in order.
#include "kernels_block.h"

namespace ssm {
namespace {

__global__ __launch_bounds__(256) void row_sums(const float* __restrict__ part, int64_t rows, int64_t width,
                                                int64_t offset, int size, int columns, float* __restrict__ to) {
  constexpr int kAhead = 8;
  __shared__ float t[16][17];
  const int col = threadIdx.x % 16, by = threadIdx.x / 16;
  const int group = blockIdx.x / columns, e = (blockIdx.x % columns) * 16 + col;
  const float* from = part + group * rows * width + offset + e;
  float x = 0.0f;
  if (e < size)
    for (int64_t r = by; r < rows; r += 16 * kAhead) {
      float v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) v[i] = r + 16 * i < rows ? from[(r + 16 * i) * width] : 0.0f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) x += v[i];
    }
  t[by][col] = x;
  __syncthreads();
  if (by != 0 || e >= size) return;
  x = 0.0f;
  for (int r = 0; r < 16; ++r) x += t[r][col];
  to[static_cast<int64_t>(group) * size + e] = x;
}

}  // namespace

hipError_t launch_row_sums(const float* part, int64_t rows_group, int groups, int64_t width, int64_t offset, int size,
                           float* to, hipStream_t stream) {
  if (!to) return hipSuccess;
  const int columns = (size + 15) / 16;
  const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(groups) * columns);
  SSM_LOG("launch row_sums: %d groups of %lld rows of %d; grid %u x 256 threads", groups,
          static_cast<long long>(rows_group), size, blocks);
  hipLaunchKernelGGL(row_sums, dim3(blocks), dim3(256), 0, stream, part, rows_group, width, offset, size, columns, to);
  return hipGetLastError();
}

}  // namespace ssm
