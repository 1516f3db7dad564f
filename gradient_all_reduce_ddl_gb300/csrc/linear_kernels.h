// linear_kernels.h -- launches of the linear layers' element-wise kernels (internal).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace ddl {

constexpr int kDzRows = 64;   // rows of dz whose column sums one CTA makes
constexpr int kMaxPlanes = 3;

// Copies a rows x cols 16-bit matrix to rows padded to ldp elements.
cudaError_t launch_pack16(const void* src, int64_t ld, void* dst, int64_t ldp, int64_t rows, int64_t cols,
                          cudaStream_t stream);

struct DzParams {
  const void* dy;
  int64_t ldy;
  const void* z;  // NULL: dz = dy
  int64_t ldz;
  int64_t rows, cols;
  int32_t type, act;
  int32_t n_planes;   // 0: column sums only
  int32_t split;      // more planes than one: binary16 halves (see plane_scale), bfloat16 thirds
  uint16_t* planes[kMaxPlanes];
  int64_t ldp;
  float* partial;     // [ceil(rows / kDzRows)][cols] column sums, or NULL
  int32_t vec;        // rows and pointers allow 4-element accesses
};
cudaError_t launch_dz(const DzParams& p, cudaStream_t stream);

// What plane k of n of dz is multiplied by.
float plane_scale(int type, int n, int k);

// db (+)= the column sums' sum, in row-block order.
cudaError_t launch_db(const float* partial, int64_t blocks, int64_t cols, void* db, int type, int accumulate,
                      cudaStream_t stream);

}  // namespace ddl
