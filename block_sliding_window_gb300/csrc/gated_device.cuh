// The activations of the MLPs: tanh-GELU of the block's own and of the gated feed-forward, and the
// latter's SiLU, each with its derivative.
#pragma once

#include "ptb_device.cuh"

namespace ptb {

__device__ __forceinline__ float gelu_tanh(float z) {
  const float k0 = 0.7978845608028654f;  // sqrt(2 / pi)
  const float k1 = 0.044715f;
  return 0.5f * z * (1.0f + tanhf(k0 * (z + k1 * z * z * z)));
}

// d/dz gelu_tanh(z) = 0.5 (1 + t) + 0.5 z (1 - t^2) c (1 + 3 a z^2),
// t = tanh(c (z + a z^3)), c = sqrt(2 / pi), a = 0.044715.
__device__ __forceinline__ float gelu_tanh_grad(float z) {
  const float k0 = 0.7978845608028654f;
  const float k1 = 0.044715f;
  const float t = tanhf(k0 * (z + k1 * z * z * z));
  return 0.5f * (1.0f + t) + 0.5f * z * (1.0f - t * t) * k0 * (1.0f + 3.0f * k1 * z * z);
}

// 1 / (1 + e^-z).  e^-z beyond fp32 gives 0, as it should.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

__device__ __forceinline__ float gated_act(float z, int act) {
  return act == kActSilu ? z * sigmoid(z) : gelu_tanh(z);
}

// act(z) and act'(z).
__device__ __forceinline__ void gated_act_grad(float z, int act, float& value, float& slope) {
  if (act == kActSilu) {
    const float s = sigmoid(z);
    value = z * s;
    slope = s * (1.f + z * (1.f - s));
  } else {
    const float k0 = 0.7978845608028654f;
    const float k1 = 0.044715f;
    const float t = tanhf(k0 * (z + k1 * z * z * z));
    value = 0.5f * z * (1.0f + t);
    slope = 0.5f * (1.0f + t) + 0.5f * z * (1.0f - t * t) * k0 * (1.0f + 3.0f * k1 * z * z);
  }
}

}  // namespace ptb
