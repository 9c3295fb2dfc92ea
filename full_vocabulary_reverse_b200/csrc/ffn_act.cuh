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
    const float phi = 0.5f * erfcf(-0.7071067811865476f * g);
    const float e = FAST ? __expf(-0.5f * g * g) : expf(-0.5f * g * g);
    *slope = fmaf(g, 0.3989422804014327f * e, phi);
    return g * phi;
  }
  if (ACT == ACT_GELU_TANH) {
    // g (1 + tanh(w)) / 2 = g sigmoid(2 w), w = sqrt(2 / pi) (g + 0.044715 g^3)
    const float q = g * g;
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
