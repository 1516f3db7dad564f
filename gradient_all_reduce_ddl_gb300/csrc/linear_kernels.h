// linear_kernels.h -- the launch before a linear layer's products (internal).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace ddl {

constexpr int kDzCols = 256;  // what a CTA makes of dz: columns, and rows by the number of them
// 64 rows where that gives work to every SM, 16 below: a small layer's pass is bound by one CTA's row loop (256 x 1000:
// 10 us with 64, 6 with 16).
inline int64_t dz_rows(int64_t rows) { return rows > 1024 ? 64 : 16; }
constexpr int kMaxPlanes = 3;

// A copy of a rows x cols 16-bit matrix with rows padded to ldp elements.
struct Pack {
  const uint16_t* src;
  int64_t ld;
  uint16_t* dst;
  int64_t ldp, rows, cols;
};

// What the products need first: up to two operand copies, and dz = dy act'(z) as planes with its column sums.
struct LinearPrep {
  int32_t n_packs;
  Pack pack[2];
  int32_t has_dz;
  const void* dy;
  int64_t ldy;
  const void* z;  // NULL: dz = dy
  int64_t ldz;
  int64_t rows, cols;
  int32_t block_rows;  // dz_rows(rows)
  int32_t type, act;
  int32_t n_planes;  // 0: column sums only
  uint16_t* planes[kMaxPlanes];
  int64_t ldp;
  int32_t vec;       // rows and pointers allow 16-byte accesses
  // the bias gradient: NULL, or db (+)= the column sums; partial has a row per dz_rows() rows, done a zero per kDzCols
  void* db;
  int32_t db_f32, accumulate;
  float* partial;
  uint32_t* done;
};
cudaError_t launch_linear_prep(const LinearPrep& p, cudaStream_t stream);

// What plane k of n of dz is multiplied by.
float plane_scale(int type, int n, int k);

}  // namespace ddl
