// ortho_kernels.h -- launches of the orthogonalised update's element-wise kernels (internal).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace ddl {

constexpr int kMaxCopies = 256;  // parameter copies of the Muon step

// A matrix of the flat buffers and its iterates' planes.
struct OrthoMatrix {
  int64_t offset, ld;  // first element, elements between rows
  int32_t rows, cols;
  uint16_t* hi[2];     // planes of the two X iterates, rows ldp elements apart
  uint16_t* lo[2];
  int64_t ldp;
  int32_t item0, n_items;  // its work items
  float shape_scale;       // sqrt(max(1, rows / cols))
  int32_t vec;             // offset, ld and cols are multiples of 4
};

// Columns [c0, c1) of rows [r0, r1) of a matrix.
struct OrthoItem {
  int32_t matrix, r0, r1, c0, c1;
};

// Elements of an item: from the largest down to the smallest, until there are two items for every SM.  A whole run of
// 64 x 147 takes 96 us (115 with the largest alone), of 2049 x 1023 276 (287), of 1000 x 2048 257 (261); with eight items
// an SM the last two take 291 and 281, since every CTA of the second pass adds all of its matrix's sums.
constexpr int kOrthoItemElems = 8192, kOrthoLeastElems = 1024, kOrthoItemsPerSm = 2;

struct OrthoPrep {
  const OrthoMatrix* matrices;
  const OrthoItem* items;
  double* partial;      // one sum of squares per item
  const void* in;       // gradient
  int32_t type;         // ElemType
  float* mom;           // NULL: the input itself is orthogonalised
  float mu;
  int32_t nesterov;
  float eps;
  int32_t n_items;
  int32_t vec;          // the buffers allow 4-element accesses
};

// v = mu v + g, and each item's sum of squares of what is orthogonalised.
cudaError_t launch_ortho_norms(const OrthoPrep& p, cudaStream_t stream);
// X = u / (|u| + eps) as planes.
cudaError_t launch_ortho_planes(const OrthoPrep& p, cudaStream_t stream);

struct OrthoFinish {
  const OrthoMatrix* matrices;
  const OrthoItem* items;
  int32_t n_items;
  int32_t iterate;      // which X holds the result
  int32_t vec;
  void* out;            // the result itself, or NULL: the parameter step
  int32_t type;
  float lr, decay;      // p = p decay - lr shape_scale x
  int32_t n_copies;
  float* copies[kMaxCopies];
};
cudaError_t launch_ortho_finish(const OrthoFinish& p, cudaStream_t stream);

}  // namespace ddl
