// xent.cuh -- the scale of the loss gradient's planes (internal).
#pragma once

#include <cstdint>

namespace ddl {

// Token t's coefficient, if it has a label and is finite, by its magnitude: as bits they order as the numbers do.
__device__ __forceinline__ uint32_t coef_bits(const float* coef, const int64_t* labels, int64_t t, int64_t vocab) {
  const int64_t y = labels[t];
  const uint32_t b = __float_as_uint(coef ? coef[t] : 1.f) & 0x7FFFFFFFu;
  return y >= 0 && y < vocab && b < 0x7F800000u ? b : 0u;
}

// What dz's planes are multiplied by, and its inverse, from the largest coefficient (of none, or of one whose inverse binary32
// does not hold, the nearest that it does).
__device__ __forceinline__ float2 dz_scale(uint32_t most, bool f16) {
  const float by = f16 ? 0x1p-14f : 1.f, top = fminf(fmaxf(__uint_as_float(most), 0x1p-100f), 0x1p100f);
  return make_float2(1.f / (top * by), top * by);
}

}  // namespace ddl
