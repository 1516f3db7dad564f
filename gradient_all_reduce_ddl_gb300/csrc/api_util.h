// api_util.h -- checks shared by the C entry points of the layer and update
// operators (internal).
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdlib>

#include "ddl.h"
#include "product.h"

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

// The arguments of a wait self-test; false if the limit is longer than the kernel's own.
inline bool give_up_of(uint32_t limit_us, uint32_t products, uint32_t loads_even, uint32_t loads_odd, GiveUp* g) {
  const uint64_t ns = (uint64_t)limit_us * 1000ull;
  if (ns > kWaitLimitNs) return false;
  *g = GiveUp{true, ns, products, {loads_even, loads_odd}};
  return true;
}

inline cudaError_t launch(const ProductLaunch& p, int tile_n, int sms, cudaStream_t stream) {
  return p.give_up.armed ? launch_product_selftest(p, tile_n, sms, stream) : launch_product(p, tile_n, sms, stream);
}

inline uint64_t round8(uint64_t n) { return (n + 7) / 8 * 8; }

// How a product is laid on the SMs: tiles of 128 x 128 on a CTA or 256 x 256 on a pair, and how many parts of the
// contraction a cluster shares out.
struct Layout {
  int tile, splits;
  double us;
};

// The layout with the least estimated time.  rounds(tile, workers): contraction steps (64-element blocks times passes)
// of the busiest of `workers` CTAs or pairs taking that tile size's tiles in turn; count(tile): tiles; shortest: blocks of
// the shortest contraction.  Measured on a GB300, in sequences of dependent launches: a step of a CTA's 128 x 128 tile
// takes 0.31 us whether one SM or all are busy (its shared memory is the bound), of a pair's 256 x 256 tile 0.28 us; the
// rest of a launch 4.3 us, 8.8 for pairs; a further tile of the same worker adds 3 and 5; joining two, four, eight parts
// 3, 3.7, 5.
template <class Rounds, class Count>
Layout choose_layout(const Rounds& rounds, const Count& count, int64_t shortest, const Residency& room) {
  Layout best{128, 1, 1e30};
  for (int tile = 128; tile <= 256; tile += 128) {
    const int width = tile / 128;
    for (int s = 1; s * width <= 8; s *= 2) {
      if (s > 1 && shortest < 2 * s) break;  // two steps each at least
      const int workers = room.clusters[s * width == 8 ? 3 : s * width / 2];
      if (workers < 1) continue;
      const int64_t waves = (count(tile) + workers - 1) / workers;
      if (s > 1 && waves > 2) break;  // many tiles: splitting only adds joins
      const double join = s == 1 ? 0.0 : s == 2 ? 3.0 : s == 4 ? 3.7 : 5.0;
      const double us = tile == 128 ? (double)rounds(128, workers) / s * 0.31 + 4.3 + join + (double)(waves - 1) * (3.0 + join)
                                    : (double)rounds(256, workers) / s * 0.28 + 8.8 + join + (double)(waves - 1) * (5.0 + join);
      if (us < best.us) best = {tile, s, us};
    }
  }
  return best;
}

}  // namespace ddl
