// activation.cuh -- the activations and their slopes, 16-bit conversions (internal).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "product.h"

namespace ddl {

__device__ __forceinline__ float from16(uint16_t u, int type) {
  return type == kBF16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}

// Two neighbours, the first in the low half.
__device__ __forceinline__ float2 from16x2(uint32_t u, int type) {
  if (type == kBF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

__device__ __forceinline__ uint16_t to16(float x, int type) {
  return type == kBF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

__device__ __forceinline__ uint32_t to16x2(float x, float y, int type) {
  uint32_t u;
  if (type == kBF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    u = *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(x, y);
    u = *reinterpret_cast<const uint32_t*>(&h);
  }
  return u;
}

// The normal distribution function Phi(z), and in *e exp(-z^2 / 2), without branches:
// Phi(-|z|) = exp(-z^2 / 2) t Q(t) with t = 1 / (1 + 0.4 |z| / sqrt 2), the form of Abramowitz & Stegun 7.1.26
// with Q of degree 8 fitted to erfcx for |z| <= 14 (Lawson's minimax iteration; relative error 6e-8, 2.2e-7
// absolute in binary32 arithmetic).
__device__ __forceinline__ float normal_cdf(float z, float* e) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = __fdividef(1.f, 1.f + 0.4f * x);
  float q = 0.0206265207f;
  q = q * t + -0.0701596215f;
  q = q * t + 0.0419936478f;
  q = q * t + 0.0439821631f;
  q = q * t + 0.0398782492f;
  q = q * t + 0.0966966003f;
  q = q * t + 0.100943796f;
  q = q * t + 0.113221556f;
  q = q * t + 0.112817116f;
  *e = __expf(-x * x);
  const float tail = q * t * *e;
  return z < 0.f ? tail : 1.f - tail;
}

__device__ __forceinline__ float activate(float z, int act) {
  float e;
  switch (act) {
    case kActRelu: return z > 0.f ? z : (z != z ? z : 0.f);
    case kActGelu: return z * normal_cdf(z, &e);
    case kActSilu: return __fdividef(z, 1.f + __expf(-z));
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.f ? 1.f : 0.f;
    case kActGelu: {
      float e;
      const float phi = normal_cdf(z, &e);
      return phi + z * (e * 0.39894228040143268f);
    }
    case kActSilu: {
      const float s = __fdividef(1.f, 1.f + __expf(-z));
      return s + z * (s * (1.f - s));
    }
    default: return 1.f;
  }
}

}  // namespace ddl
