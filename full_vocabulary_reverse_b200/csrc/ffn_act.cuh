// ffn_act.cuh -- the gated block's activations act(g) and their derivatives.
// FAST takes the hardware's exponential and reciprocal (relative error about
// 2^-21 for the magnitudes that matter): enough in front of a rounding to
// bf16, not for fp32 results.
#pragma once

#include <cuda_runtime.h>

namespace rkl {

enum : int { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2, ACT_RELU = 3 };

template <bool FAST>
__device__ __forceinline__ float act_sigmoid(float x) {
  if (FAST) return __fdividef(1.f, 1.f + __expf(-x));
  return 1.f / (1.f + expf(-x));
}

// erfc(z) / 2 for z >= 0 by the Chebyshev fit t exp(-z^2 + P(t)), t = 1 / (1 +
// z / 2), of Press, Teukolsky, Vetterling and Flannery, "Numerical Recipes"
// (relative error 1.2e-7 for all z): about 16 instructions, a third of erfcf's.
__device__ __forceinline__ float half_erfc_fit(float z) {
  float t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.5f, z, 1.f)));
  float p = 0.17087277f;
  p = fmaf(p, t, -0.82215223f);
  p = fmaf(p, t, 1.48851587f);
  p = fmaf(p, t, -1.13520398f);
  p = fmaf(p, t, 0.27886807f);
  p = fmaf(p, t, -0.18628806f);
  p = fmaf(p, t, 0.09678418f);
  p = fmaf(p, t, 0.37409196f);
  p = fmaf(p, t, 1.00002368f);
  p = fmaf(p, t, -1.26551223f);
  return 0.5f * t * __expf(fmaf(-z, z, p));
}

// act(g), and in *slope its derivative.
template <int ACT, bool FAST>
__device__ __forceinline__ float act_with_slope(float g, float* slope) {
  if (ACT == ACT_SILU) {
    const float s = act_sigmoid<FAST>(g);
    *slope = s * fmaf(g, 1.f - s, 1.f);
    return g * s;
  }
  if (ACT == ACT_GELU) {
    // g Phi(g), Phi = erfc(-g / sqrt(2)) / 2: no cancellation for negative g
    float phi;
    if (FAST) {
      const float tail = half_erfc_fit(0.7071067811865476f * fabsf(g));  // Phi(-|g|)
      phi = g < 0.f ? tail : 1.f - tail;
    } else {
      phi = 0.5f * erfcf(-0.7071067811865476f * g);
    }
    const float e = FAST ? __expf(-0.5f * g * g) : expf(-0.5f * g * g);
    *slope = fmaf(g, 0.3989422804014327f * e, phi);
    return g * phi;
  }
  if (ACT == ACT_GELU_TANH) {
    // g (1 + tanh(w)) / 2 = g sigmoid(2 w), w = sqrt(2 / pi) (g + 0.044715 g^3)
    // (far out s is 0 or 1 and s (1 - s) 0; a finite g^2 keeps 0 x infinity out of the slope)
    const float q = fminf(g * g, 1e12f);
    const float s = act_sigmoid<FAST>(1.5957691216057308f * g * fmaf(0.044715f, q, 1.f));
    *slope = fmaf(s * (1.f - s) * g, 1.5957691216057308f * fmaf(0.134145f, q, 1.f), s);
    return g * s;
  }
  *slope = g > 0.f ? 1.f : 0.f;
  return g > 0.f || g != g ? g : 0.f;
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act_only(float g) {
  float slope;
  return act_with_slope<ACT, FAST>(g, &slope);
}

}  // namespace rkl
