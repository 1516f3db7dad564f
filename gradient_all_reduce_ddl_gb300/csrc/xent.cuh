// xent.cuh -- the scale of the loss gradient's planes (internal).
#pragma once

#include <cstdint>

namespace ddl {

// Token t's coefficient, if it has a label and is finite, by its magnitude: as bits they order as the numbers do.  0: the token
// does not count.
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

// Binary32 dw of a bfloat16 head takes dz in three planes (24 bits) where at most so many tokens count, else in two.  Two leave
// it 1.5 to 2.4e-6 off however many there are.  Sums in binary32 lose 1.9e-8 times the root of the number of tokens that
// are not zero (2112: 0.7e-6, 4096: 1.2e-6, 8192: 1.75e-6), about as much from here on, while a third pass costs a fifth of the
// products (6000 tokens, 2048 features, 65,536 entries: 4330 -> 5500 us backward; 8192: 7760 -> 9280 with the loss, 1.6e-6 ->
// 0.7e-6 off).
constexpr uint32_t kExactTokens = 4096;
__device__ __forceinline__ int planes_of(uint32_t counted, int most) { return most == 3 && counted > kExactTokens ? 2 : most; }

}  // namespace ddl
