// The walk over the chunks (delta_walk.h) for bfloat16 inputs whose rows load straight into LDS.
#include "delta_walk.h"

namespace ssm {

hipError_t launch_walk_bf16_direct(const DeltaPlan& p, const DeltaChunks& plan, const ScanArgs& s, hipStream_t stream) {
  return launch_all<bf16_t, 1, true>(p, plan, s, stream);
}

}  // namespace ssm
