// The gate of a gated feed-forward projection: h = act(g) u, and its
// derivatives, in fp32.
#pragma once
#include "common.cuh"
#include "f32x2.cuh"

namespace mlpk {

constexpr int ACT_SILU = 3;   // g / (1 + e^{-g}); the gated operations only

constexpr float kLog2e = 1.4426950408889634f;

// max(g, 0); NaN stays NaN (fmaxf would return 0 and hide a broken gate).
__device__ __forceinline__ float gate_relu(float g) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(g));
  return r;
}
__device__ __forceinline__ float gate_act(float g, int act) {
  if (act == ACT_RELU) return gate_relu(g);
  if (act == ACT_SILU) return g * rcp_fast(1.0f + ex2_fast(-kLog2e * g));
  return apply_act(g, act);
}
// act(g) and act'(g) together.  Both smooth activations are g s with s =
// 1 / (1 + e): for SiLU e = e^{-g}, for GELU (tanh form) e = e^{-2a}
// (common.cuh), and 1 - s = e s keeps its relative accuracy in the tails.  The
// gate is clamped where e would leave 2^-126 .. 2^126 (SiLU: 87.3, GELU: 10):
// act' has reached 1 there, or 0 but for 2^-118, while e (s) held at its bound
// would still be multiplied by g (GELU: g^3).  Beyond, act is g, or 0 but for 2^-119.
__device__ __forceinline__ void gate_act_grad(float g, int act, float& a, float& da) {
  if (act == ACT_RELU) {
    a = gate_relu(g);
    da = g > 0.0f ? 1.0f : 0.0f;
  } else if (act == ACT_GELU_TANH) {
    const float c = clamp_abs(g, 10.0f);
    const float g2 = c * c;
    const float e = ex2_fast(c * fmaf(kGeluC1, g2, kGeluC0));
    const float s = rcp_fast(1.0f + e);
    a = (g < c ? c : g) * s;
    da = fmaf(2.0f * (c * s) * (e * s), fmaf(kGeluK3, g2, kGeluK0), s);
  } else if (act == ACT_SILU) {
    const float c = clamp_abs(g, 87.3f);
    const float e = ex2_fast(-kLog2e * c);
    const float s = rcp_fast(1.0f + e);
    a = (g < c ? c : g) * s;
    da = fmaf(c * s, e * s, s);
  } else {
    a = g;
    da = 1.0f;
  }
}

// The same for two gates whose results are rounded to bf16.  1 - s stands for
// e s here: off by 2^-24 where s is near 1, which GELU's other factor (35 at g =
// 5) makes 2e-6 of act' at most; from g = 6 on 1 - s is 0.  With no clamp of e an
// infinite one leaves s = 0, a = -0, act' = 0; in act' g^2 is held at 256, so that
// 1 - s = 0 or a = 0 meets no infinity.
template <int ACT>
__device__ __forceinline__ void gate2(F2 g, F2& a, F2& da) {
  if constexpr (ACT == ACT_NONE) {
    a = g;
    da = pack2(1.0f, 1.0f);
  } else if constexpr (ACT == ACT_RELU) {
    float x, y;
    unpack2(g, x, y);
    a = pack2(gate_relu(x), gate_relu(y));
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
    unpack2(g2, x0, x1);
    const F2 near2 = pack2(fminf(x0, 256.f), fminf(x1, 256.f));
    da = ACT == ACT_SILU
             ? fma2(a, rest, s)
             : fma2(mul2(a, rest), fma2(near2, pack2(2 * kGeluK3, 2 * kGeluK3), pack2(2 * kGeluK0, 2 * kGeluK0)), s);
  }
}

}  // namespace mlpk
