// Picks the instance of a gated linear recurrence kernel for a call's types:
// F::run<InT, DECAY, MIX>(arguments...).
#pragma once

#include <utility>

#include "device_math.h"
#include "kernels_glr.h"

namespace ssm {

template <typename F, typename InT, int DECAY, typename... X>
hipError_t glr_pick_mix(int mix, X&&... x) {
  if (mix == kGlrUnit) return F::template run<InT, DECAY, kGlrUnit>(std::forward<X>(x)...);
  if (mix == kGlrRest) return F::template run<InT, DECAY, kGlrRest>(std::forward<X>(x)...);
  return F::template run<InT, DECAY, kGlrOne>(std::forward<X>(x)...);
}

template <typename F, typename... X>
hipError_t glr_pick(const GlrPlan& p, X&&... x) {
  if (p.in_bf16)
    return p.decay == kGlrSigmoid ? glr_pick_mix<F, bf16_t, kGlrSigmoid>(p.mix, std::forward<X>(x)...)
                                  : glr_pick_mix<F, bf16_t, kGlrSoftplus>(p.mix, std::forward<X>(x)...);
  return p.decay == kGlrSigmoid ? glr_pick_mix<F, float, kGlrSigmoid>(p.mix, std::forward<X>(x)...)
                                : glr_pick_mix<F, float, kGlrSoftplus>(p.mix, std::forward<X>(x)...);
}

}  // namespace ssm
