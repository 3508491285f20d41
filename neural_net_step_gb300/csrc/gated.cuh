// The gate of a gated feed-forward projection: h = act(g) u, and its
// derivatives, in fp32.
#pragma once
#include "common.cuh"

namespace mlpk {

constexpr int ACT_SILU = 3;   // g / (1 + e^{-g}); the gated operations only

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float gate_act(float g, int act) {
  if (act == ACT_SILU) return g * rcp_fast(1.0f + ex2_fast(-kLog2e * g));
  return apply_act(g, act);
}
// act(g) and act'(g) together.  Both smooth activations are g s with s =
// 1 / (1 + e): for SiLU e = e^{-g}, for GELU (tanh form) e = e^{-2a}
// (common.cuh); the exponent is clamped so that e stays finite, and 1 - s =
// e s keeps its relative accuracy in the tails.
__device__ __forceinline__ void gate_act_grad(float g, int act, float& a, float& da) {
  if (act == ACT_RELU) {
    a = fmaxf(g, 0.0f);
    da = g > 0.0f ? 1.0f : 0.0f;
  } else if (act == ACT_GELU_TANH) {
    const float g2 = g * g;
    const float e = ex2_fast(fminf(fmaxf(g * fmaf(kGeluC1, g2, kGeluC0), -126.f), 126.f));
    const float s = rcp_fast(1.0f + e);
    a = g * s;
    da = fmaf(2.0f * a * (e * s), fmaf(kGeluK3, g2, kGeluK0), s);
  } else if (act == ACT_SILU) {
    const float e = ex2_fast(fminf(-kLog2e * g, 126.f));
    const float s = rcp_fast(1.0f + e);
    a = g * s;
    da = fmaf(a, e * s, s);
  } else {
    a = g;
    da = 1.0f;
  }
}

}  // namespace mlpk
