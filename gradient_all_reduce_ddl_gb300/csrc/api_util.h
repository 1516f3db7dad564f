// api_util.h -- checks shared by the C entry points of the layer and update
// operators (internal).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>

#include "ddl.h"

namespace ddl {

inline ddl_status_t status_of(cudaError_t e) {
  if (e == cudaSuccess) return DDL_OK;
  cudaGetLastError();  // clear a non-sticky error so later calls start clean
  return e == cudaErrorMemoryAllocation ? DDL_ERR_OOM : DDL_ERR_CUDA;
}

// DDL_INJECT_ALLOC_FAILURE=1: device allocations fail as if memory were short.
inline cudaError_t device_alloc(void** p, size_t bytes) {
  const char* v = std::getenv("DDL_INJECT_ALLOC_FAILURE");
  if (v && v[0] == '1' && v[1] == '\0') return cudaErrorMemoryAllocation;
  return cudaMalloc(p, bytes);
}

// Memory that a kernel on `device` may use as a caller's buffer.
inline bool device_pointer(const void* p, int device) {
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return at.type == cudaMemoryTypeManaged || (at.type == cudaMemoryTypeDevice && at.device == device);
}

// Byte range of a buffer; empty ranges overlap nothing.
struct Range {
  uintptr_t lo, hi;
  Range(const void* p, uint64_t bytes) : lo(reinterpret_cast<uintptr_t>(p)), hi(p ? lo + bytes : lo) {}
  bool overlaps(const Range& o) const { return lo < o.hi && o.lo < hi; }
  bool wraps() const { return hi < lo; }
};

inline uint64_t round8(uint64_t n) { return (n + 7) / 8 * 8; }

// CTAs per cluster for `tiles` tiles of a contraction of `blocks` K blocks:
// doubled while the doubled clusters still fit on the SMs and leave each CTA
// two K blocks.
inline int choose_splits(int64_t tiles, int64_t blocks, int sms) {
  int s = 1;
  while (s < 8 && tiles * s * 2 <= sms && blocks >= 4 * s) s *= 2;
  return s;
}

// Whether a product of `tiles128` 128 x 128 tiles runs faster as `tiles256` 256 x 256 tiles on CTA pairs: both sides'
// rounds over the SMs, a pair's tile being twice a CTA's work at 1 / kPairGain of its time.
constexpr double kPairGain = 1.7;
inline bool prefer_pairs(int64_t tiles128, int64_t tiles256, int sms) {
  const int64_t rounds128 = (tiles128 + sms - 1) / sms, rounds256 = (tiles256 + sms / 2 - 1) / (sms / 2);
  return tiles128 > sms / 2 && (double)rounds256 * 2.0 < (double)rounds128 * kPairGain;
}

}  // namespace ddl
