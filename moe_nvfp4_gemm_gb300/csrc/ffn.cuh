// Shared by the kernels of the gated feed-forward block: 16-bit values and the activations.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace nvfp4 {

// Two fp32 values rounded to bf16 or fp16, `lo` in the low half.
template <bool HALF>
DEVI uint32_t pack16(float lo, float hi) {
  if (!HALF) return pack_bf16x2(lo, hi);
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool HALF>
DEVI float unpack16(uint32_t w, int which) {
  if (!HALF) return __uint_as_float(which ? w & 0xFFFF0000u : w << 16);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(which ? w >> 16 : w & 0xFFFFu)));
}

// sigma(x) = 1 / (1 + exp(-x)) by the fast exponential and division: a few parts in 10^7 (10^-6 at x = -20),
// far below a step of the 16-bit results. exp(-x) past the type's range gives 0.
DEVI float ffn_sigmoid(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

constexpr float kGeluScale = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// act(g) = g sigma(p(g)); act 0: silu, p = g; act 1: gelu in its tanh form, as 0.5 (1 + tanh(v)) = sigma(2 v).
DEVI float ffn_act(float g, int act) {
  const float p = act == 0 ? g : kGeluScale * (g + kGeluCubic * g * g * g);
  return g * ffn_sigmoid(p);
}

// act(g) and its derivative sigma + g sigma (1 - sigma) p'(g). For |g| > 100 the factor sigma (1 - sigma) is 0
// in gelu; bounding g there keeps p' finite, so that the product is 0 and not NaN.
DEVI void ffn_act_grad(float g, int act, float& a, float& slope) {
  const float p = act == 0 ? g : kGeluScale * (g + kGeluCubic * g * g * g);
  const float s = ffn_sigmoid(p);
  a = g * s;
  float dp = 1.0f;
  if (act != 0) {
    const float b = fminf(fabsf(g), 100.0f);
    dp = kGeluScale * (1.0f + 3.0f * kGeluCubic * b * b);
  }
  slope = s + a * (1.0f - s) * dp;
}

}  // namespace nvfp4
