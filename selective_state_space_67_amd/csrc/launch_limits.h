// The largest grid of one launch. Plain host arithmetic.
#pragma once

#include <stdint.h>

namespace ssm {

// A launch's threads are counted in 32 bits. With more of them it fails, or goes through with
// the rest of the division by 2^32 only and no error.
inline bool fits_launch(int64_t blocks, int64_t threads) { return blocks <= ((int64_t{1} << 32) - 1) / threads; }

}  // namespace ssm
