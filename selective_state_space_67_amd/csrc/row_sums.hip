// Sums over the workgroups' rows of partial sums (parameters' gradients of the norms
// around a block and of the gated linear recurrence): 32 columns a workgroup (a row's
// 128 bytes at a time: 512 rows of 4608 sums 4.8 us, with 16 columns 6.6, with 64
// 5.7), 32 threads a column, each adding every 32nd row in order with eight of them
// under way, then the 32 sums in order. Up to three sums go in one launch, unless together
// they have more workgroups than one has room for.
#include "kernels_block.h"

namespace ssm {
namespace {

struct SumsArgs {
  RowSum sum[3];
  int first[4];  // workgroup that each starts with
  int64_t width;
  int size, columns;
};

constexpr int kCols = 32, kBy = 32;  // columns, threads a column

__global__ __launch_bounds__(kCols * kBy) void row_sums(const float* __restrict__ part, const SumsArgs a) {
  constexpr int kAhead = 8;
  __shared__ float t[kBy][kCols + 1];
  const int block = blockIdx.x, which = block >= a.first[2] ? 2 : block >= a.first[1] ? 1 : 0;
  const RowSum& s = a.sum[which];
  const int mine = block - a.first[which], group = mine / a.columns;
  const int col = threadIdx.x % kCols, by = threadIdx.x / kCols, e = (mine - group * a.columns) * kCols + col;
  const float* from = part + group * s.rows_group * a.width + s.offset + e;
  float x = 0.0f;
  if (e < a.size)
    for (int64_t r = by; r < s.rows_group; r += kBy * kAhead) {
      float v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) v[i] = r + kBy * i < s.rows_group ? from[(r + kBy * i) * a.width] : 0.0f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) x += v[i];
    }
  t[by][col] = x;
  __syncthreads();
  if (by != 0 || e >= a.size) return;
  x = 0.0f;
  for (int r = 0; r < kBy; ++r) x += t[r][col];
  s.to[static_cast<int64_t>(group) * a.size + e] = x;
}

}  // namespace

hipError_t launch_row_sums(const float* part, int64_t width, int size, const RowSum (&sums)[3], hipStream_t stream) {
  const int columns = (size + kCols - 1) / kCols;
  int64_t total = 0;
  int n = 0;
  for (const RowSum& s : sums)
    if (s.to) {
      total += static_cast<int64_t>(s.groups) * columns;
      ++n;
    }
  if (n == 0) return hipSuccess;
  if (!fits_launch(total, kCols * kBy)) {  // (a gate for each of very many sequences, and the weights)
    if (n == 1) return hipErrorInvalidConfiguration;
    hipError_t e = hipSuccess;
    for (const RowSum& s : sums)
      if (e == hipSuccess) e = launch_row_sums(part, width, size, {s, {}, {}}, stream);
    return e;
  }
  SumsArgs a{};
  a.width = width;
  a.size = size;
  a.columns = columns;
  n = 0;
  unsigned blocks = 0;
  for (const RowSum& s : sums)
    if (s.to) {
      a.first[n] = static_cast<int>(blocks);
      a.sum[n++] = s;
      blocks += static_cast<unsigned>(s.groups) * columns;
    }
  for (int i = n; i < 4; ++i) a.first[i] = 0x7fffffff;
  SSM_LOG("launch row_sums: %d sums of rows of %d; grid %u x %d threads", n, size, blocks, kCols * kBy);
  hipLaunchKernelGGL(row_sums, dim3(blocks), dim3(kCols * kBy), 0, stream, part, a);
  return hipGetLastError();
}

}  // namespace ssm
