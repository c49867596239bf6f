// Picks the instance of a gated linear recurrence kernel for a call's types and
// options: F::run<InT, DECAY, MIX, IN, Z>(arguments...), with IN an input gate and Z
// an output gate.
#pragma once

#include <utility>

#include "device_math.h"
#include "kernels_glr.h"

namespace ssm {

template <typename F, typename InT, int DECAY, int MIX, typename... X>
hipError_t glr_pick_gates(const GlrPlan& p, X&&... x) {
  if (p.in)
    return p.z ? F::template run<InT, DECAY, MIX, true, true>(std::forward<X>(x)...)
               : F::template run<InT, DECAY, MIX, true, false>(std::forward<X>(x)...);
  return p.z ? F::template run<InT, DECAY, MIX, false, true>(std::forward<X>(x)...)
             : F::template run<InT, DECAY, MIX, false, false>(std::forward<X>(x)...);
}

template <typename F, typename InT, int DECAY, typename... X>
hipError_t glr_pick_mix(const GlrPlan& p, X&&... x) {
  if (p.mix == kGlrUnit) return glr_pick_gates<F, InT, DECAY, kGlrUnit>(p, std::forward<X>(x)...);
  if (p.mix == kGlrRest) return glr_pick_gates<F, InT, DECAY, kGlrRest>(p, std::forward<X>(x)...);
  return glr_pick_gates<F, InT, DECAY, kGlrOne>(p, std::forward<X>(x)...);
}

template <typename F, typename... X>
hipError_t glr_pick(const GlrPlan& p, X&&... x) {
  if (p.in_bf16)
    return p.decay == kGlrSigmoid ? glr_pick_mix<F, bf16_t, kGlrSigmoid>(p, std::forward<X>(x)...)
                                  : glr_pick_mix<F, bf16_t, kGlrSoftplus>(p, std::forward<X>(x)...);
  return p.decay == kGlrSigmoid ? glr_pick_mix<F, float, kGlrSigmoid>(p, std::forward<X>(x)...)
                                : glr_pick_mix<F, float, kGlrSoftplus>(p, std::forward<X>(x)...);
}

}  // namespace ssm
