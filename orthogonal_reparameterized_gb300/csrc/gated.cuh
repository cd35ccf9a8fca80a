// The activation of the gated feed-forward block: a(g) = g s(t), s(t) = 1 / (1 + exp(-t)).
#pragma once

#include "common.cuh"

namespace poetx {

// t = g (c0 + c1 g^2): SiLU 1 and 0, GELU 2 sqrt(2 / pi) and 0.044715 times that.
struct Act {
  float c0, c1;
};
inline Act act_of(poetx_activation a) {
  const double c = 1.5957691216057307117;  // 2 sqrt(2 / pi)
  return a == POETX_GELU ? Act{(float)c, (float)(0.044715 * c)} : Act{1.f, 0.f};
}
inline bool act_ok(poetx_activation a) { return a == POETX_SILU || a == POETX_GELU; }

// s(t).  EXACT: for fp32 results.  Otherwise the hardware's exp2 and reciprocal, each within 2^-22; the
// argument's rounding costs |t| 2^-24 besides (exp(-t) at t = -80: 5e-6), all far below bf16's 2^-8.
template <bool EXACT>
__device__ __forceinline__ float logistic(float t) {
  if (EXACT) return 1.f / (1.f + expf(-t));
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t * -1.44269504088896340736f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
// g^2, cut off where fp32 ends (0 times infinity would make SiLU's t NaN).
__device__ __forceinline__ float square(float g) { return fminf(g * g, 0x1p120f); }

template <bool EXACT>
__device__ __forceinline__ float gated(float g, float u, Act a) {
  return g * logistic<EXACT>(g * fmaf(a.c1, square(g), a.c0)) * u;
}
// (dg, du) of dh.
template <bool EXACT>
__device__ __forceinline__ float2 gated_grad(float g, float u, float dh, Act a) {
  const float q = square(g);
  const float s = logistic<EXACT>(g * fmaf(a.c1, q, a.c0));
  const float v = g * s;
  const float d = fmaf(v * (1.f - s), fmaf(3.f * a.c1, q, a.c0), s);
  return make_float2(dh * u * d, dh * v);
}

// What is left of v after its rounding to bf16, which is v's first piece (nothing, where that is not finite).
__device__ __forceinline__ float rest_of(float v, __nv_bfloat16 first) {
  const float f = __bfloat162float(first);
  return isfinite(f) ? v - f : 0.f;
}

}  // namespace poetx
