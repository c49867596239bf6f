// The walk over the chunks (delta_walk.h) for float32 inputs.
#include "delta_walk.h"

namespace ssm {

hipError_t launch_walk_f32(const DeltaPlan& p, const DeltaChunks& plan, const ScanArgs& s, hipStream_t stream) {
  return launch_all<float, 3, false>(p, plan, s, stream);
}

}  // namespace ssm
