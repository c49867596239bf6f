// Threads of the scan kernels' workgroups, for the front end's check of their grids.
#include "scan_fwd_kernel.h"

namespace ssm {

int scan_block_threads(int64_t N) {
  int threads = 0;
  (void)fwd::with_tile(N, [&](auto tile) {
    threads = decltype(tile)::THREADS;
    return hipSuccess;
  });
  return threads;
}

}  // namespace ssm
