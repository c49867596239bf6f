// The walk over the chunks (delta_walk.h) for other bfloat16 inputs (odd sizes, strides or addresses).
#include "delta_walk.h"

namespace ssm {

hipError_t launch_walk_bf16(const DeltaPlan& p, const DeltaChunks& plan, const ScanArgs& s, hipStream_t stream) {
  return launch_all<bf16_t, 1, false>(p, plan, s, stream);
}

}  // namespace ssm
