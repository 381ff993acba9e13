// The activations of a gated feed-forward, SiLU and tanh-GELU, with their derivatives.
//
// Both are z sigma(w) with w = z (c0 + c1 z^2): c0 = 1, c1 = 0 for SiLU, and since
// (1 + tanh v) / 2 = sigma(2 v), c0 = 2 sqrt(2 / pi), c1 = 0.044715 c0 for the tanh-GELU.  One
// formula without a branch keeps the epilogues' unrolled code small, and sigma keeps its relative
// precision where 1 + tanh cancels.  The derivative is sigma + z sigma (1 - sigma) w'.
#pragma once

#include "ptb_device.cuh"

namespace ptb {

struct GatedAct {
  float c0, c1;
  __device__ explicit GatedAct(int act)
      : c0(act == kActSilu ? 1.f : 1.5957691216057308f),
        c1(act == kActSilu ? 0.f : 0.071354816272600250f) {}

  // z^2, kept finite so that c1 = 0 cannot meet an infinity.
  static __device__ __forceinline__ float square(float z) { return fminf(z * z, 1e30f); }

  // 1 / (1 + e^-w); e^-w beyond fp32 gives 0, as it should.
  static __device__ __forceinline__ float sigmoid(float w) {
    return __fdividef(1.f, 1.f + __expf(-w));
  }

  __device__ __forceinline__ float value(float z) const {
    return z * sigmoid(z * fmaf(c1, square(z), c0));
  }

  __device__ __forceinline__ void value_and_slope(float z, float& v, float& slope) const {
    const float q = square(z);
    const float s = sigmoid(z * fmaf(c1, q, c0));
    v = z * s;
    slope = fmaf(v * (1.f - s), fmaf(3.f * c1, q, c0), s);
  }
};

}  // namespace ptb
