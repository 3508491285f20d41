// The gate of a gated feed-forward projection: h = act(g) u, and its
// derivatives, in fp32.
#pragma once
#include "common.cuh"
#include "f32x2.cuh"

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

// The same for two gates whose results are rounded to bf16.  1 - s stands for
// e s here: off by 2^-24 where s is near 1 (act' is too), and with no clamp an
// infinite e leaves s = 0, a = -0, act' = -0.
template <int ACT>
__device__ __forceinline__ void gate2(F2 g, F2& a, F2& da) {
  if constexpr (ACT == ACT_NONE) {
    a = g;
    da = pack2(1.0f, 1.0f);
  } else if constexpr (ACT == ACT_RELU) {
    float x, y;
    unpack2(g, x, y);
    a = pack2(fmaxf(x, 0.0f), fmaxf(y, 0.0f));
    da = pack2(x > 0.0f ? 1.0f : 0.0f, y > 0.0f ? 1.0f : 0.0f);
  } else {
    const F2 one = pack2(1.0f, 1.0f), minus = pack2(-1.0f, -1.0f);
    const F2 g2 = mul2(g, g);
    const F2 x = ACT == ACT_SILU ? mul2(g, pack2(-kLog2e, -kLog2e))
                                 : mul2(g, fma2(g2, pack2(kGeluC1, kGeluC1), pack2(kGeluC0, kGeluC0)));
    float x0, x1;
    unpack2(x, x0, x1);
    unpack2(add2(pack2(ex2_fast(x0), ex2_fast(x1)), one), x0, x1);
    const F2 s = pack2(rcp_fast(x0), rcp_fast(x1));
    a = mul2(g, s);
    const F2 rest = fma2(s, minus, one);   // 1 - s
    da = ACT == ACT_SILU
             ? fma2(a, rest, s)
             : fma2(mul2(a, rest), fma2(g2, pack2(2 * kGeluK3, 2 * kGeluK3), pack2(2 * kGeluK0, 2 * kGeluK0)), s);
  }
}

}  // namespace mlpk
