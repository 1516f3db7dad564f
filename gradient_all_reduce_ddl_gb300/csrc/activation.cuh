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

// Two binary32 numbers in one register pair: half the instructions of what bounds an epilogue.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void from_pair(uint64_t d, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(d));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// N activations whose results will be rounded to 16 bits.
// GELU: z Phi(z) with Phi(-|z|) = 2^P(|z|), P of degree 11 fitted to the binary logarithm of Phi(-x) for x <= 14.4, where
// 2^P is zero (Lawson's minimax iteration).  In binary32 arithmetic it is 6.4e-7 off at most (|z| between 1 and 3), and
// 2e-5 relative for |z| <= 5.5, where half a unit in the last place of binary16 is 2.4e-4.  One exponential and eleven half
// multiply-adds a value: the function unit, at 16 values a cycle and SM, and the issue slots are about equally busy.
template <int ACT, int N>
__device__ __forceinline__ void activate(float (&v)[N]) {
  static_assert(N % 2 == 0);
  if constexpr (ACT == kActRelu) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = v[k] > 0.f ? v[k] : (v[k] != v[k] ? v[k] : 0.f);
  } else if constexpr (ACT == kActGelu) {
    constexpr float kP[12] = {-0.999999106f,    -1.15114534f,     -0.458924085f,   -0.0532146543f, 0.007907358f,    -0.000652429822f,
                              -1.80448078e-05f, 1.26337518e-05f, -1.64435778e-06f, 1.10605363e-07f, -3.93015087e-09f, 5.83025503e-11f};
    uint64_t x[N / 2], q[N / 2];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      x[k] = pair_of(fminf(fabsf(v[2 * k]), 14.4f), fminf(fabsf(v[2 * k + 1]), 14.4f));
      q[k] = pair_of(kP[11], kP[11]);
    }
#pragma unroll
    for (int i = 10; i >= 0; --i) {
      const uint64_t c = pair_of(kP[i], kP[i]);
#pragma unroll
      for (int k = 0; k < N / 2; ++k) q[k] = fma_pair(q[k], x[k], c);
    }
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      float a, b, c, d;
      from_pair(q[k], &a, &b);
      a = exp2_fast(a), b = exp2_fast(b);
      from_pair(fma_pair(pair_of(a, b), pair_of(-1.f, -1.f), pair_of(1.f, 1.f)), &c, &d);
      const uint64_t phi = pair_of(v[2 * k] < 0.f ? a : c, v[2 * k + 1] < 0.f ? b : d);
      from_pair(mul_pair(pair_of(v[2 * k], v[2 * k + 1]), phi), &v[2 * k], &v[2 * k + 1]);
    }
  } else if constexpr (ACT == kActSilu) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] *= rcp_fast(1.f + exp2_fast(-1.4426950408889634f * v[k]));
  }
}

template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  switch (act) {
    case kActRelu: activate<kActRelu>(v); break;
    case kActGelu: activate<kActGelu>(v); break;
    case kActSilu: activate<kActSilu>(v); break;
    default: break;
  }
}

// The normal distribution function Phi(z), and in *e exp(-z^2 / 2), without branches:
// Phi(-|z|) = exp(-z^2 / 2) t Q(t) with t = 1 / (1 + 0.4 |z| / sqrt 2), the form of Abramowitz & Stegun 7.1.26
// with Q of degree 8 fitted to erfcx for |z| <= 14 (Lawson's minimax iteration; relative error 6e-8, 2.2e-7
// absolute in binary32 arithmetic).
__device__ __forceinline__ float normal_cdf(float z, float* e) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = rcp_fast(1.f + 0.4f * x);
  float q = 0.0206265207f;
  q = q * t + -0.0701596215f;
  q = q * t + 0.0419936478f;
  q = q * t + 0.0439821631f;
  q = q * t + 0.0398782492f;
  q = q * t + 0.0966966003f;
  q = q * t + 0.100943796f;
  q = q * t + 0.113221556f;
  q = q * t + 0.112817116f;
  *e = exp2_fast(z * z * -0.72134752044448170f);  // -log2(e) / 2
  const float tail = q * t * *e;
  return z < 0.f ? tail : 1.f - tail;
}

// The slopes that dy is multiplied by (ReLU's selects instead).
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case kActGelu: {
      float e;
      const float phi = normal_cdf(z, &e);
      return phi + z * (e * 0.39894228040143268f);
    }
    case kActSilu: {
      const float s = rcp_fast(1.f + exp2_fast(-1.4426950408889634f * z));
      return s + z * (s * (1.f - s));
    }
    default: return 1.f;
  }
}

}  // namespace ddl
