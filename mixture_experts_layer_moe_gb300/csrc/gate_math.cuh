// The SwiGLU gate and its gradient in fp32, as the tensor-core paths form them
// (hardware exp and division, within 2^-17 of the value), and bf16 bits.
#pragma once

#include "common.cuh"

namespace moe {

__device__ __forceinline__ float silu_mul(float a, float b) {
  return __fdividef(a, 1.f + __expf(-a)) * b;
}

// With s = 1 / (1 + e^-g):  dg = dh u s (1 + g (1 - s)),  du = dh g s.
__device__ __forceinline__ void swiglu_grad(float dh, float g, float u, float &dg, float &du) {
  const float s = __fdividef(1.f, 1.f + __expf(-g));
  dg = dh * u * s * (1.f + g * (1.f - s));
  du = dh * g * s;
}

__device__ __forceinline__ float bf16_value(uint16_t b) {
  return __uint_as_float((uint32_t)b << 16);
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t *>(&h);
}

}  // namespace moe
