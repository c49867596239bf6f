// Sums over groups of consecutive lanes (gfx950).
#pragma once

#include <hip/hip_runtime.h>

namespace ssm {

// Sum over LR consecutive lanes (a power of two), in all of them.
template <int CTRL>
__device__ __forceinline__ float dpp_all(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}
template <int LR>
__device__ __forceinline__ float lanes_sum(float x) {
  if constexpr (LR >= 2) x = dpp_all<0xB1>(x);    // quad_perm 1,0,3,2
  if constexpr (LR >= 4) x = dpp_all<0x4E>(x);    // quad_perm 2,3,0,1
  if constexpr (LR >= 8) x = dpp_all<0x141>(x);   // row_half_mirror
  if constexpr (LR >= 16) x = dpp_all<0x140>(x);  // row_mirror
  if constexpr (LR >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if constexpr (LR >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return x;
}

}  // namespace ssm
