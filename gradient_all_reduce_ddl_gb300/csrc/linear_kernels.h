// linear_kernels.h -- the launch before a linear layer's products (internal).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace ddl {

constexpr int kDzCols = 256;  // what a CTA makes of dz: columns, and rows by the number of them
// Few rows: 16 a CTA, whose row loop bounds a small pass; more: 64, which leaves fewer sums to add at the end.  Column
// sums of a GELU layer's dz, 16 against 64 rows: 1024 x 128 6.5 and 7.8 us, 1024 x 4096 11.4 and 12.4, 2048 x 128 9.2
// and 8.0, 2048 x 4096 19.0 and 13.8, 8192 x 8192 126 and 78.
constexpr int64_t kDzFewRows = 1024;
inline int64_t dz_rows(int64_t rows) { return rows > kDzFewRows ? 64 : 16; }
// The most row blocks of a pass over up to `most` rows, for the workspace of their sums.
inline int64_t dz_row_blocks(int64_t most) {
  const int64_t few = most < kDzFewRows ? most : kDzFewRows, a = (few + 15) / 16, b = (most + 63) / 64;
  return a > b ? a : b;
}
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
