// ortho_kernels.h -- launches of the Newton-Schulz steps' element-wise kernels (internal).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace ddl {

// A matrix of the flat buffers and its first iterate's planes.
struct OrthoMatrix {
  int64_t offset, ld;   // first element, elements between rows
  int64_t rows, cols;
  uint16_t* hi;         // planes of X, rows ldp elements apart
  uint16_t* lo;
  int64_t ldp;
  int32_t item0, n_items;  // its work items
};

// Elements [begin, end) of a matrix's row-major order.
struct OrthoItem {
  int32_t matrix, pad;
  int64_t begin, end;
};

constexpr int kOrthoItemElems = 8192;

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
};

// v = mu v + g, and each item's sum of squares of what is orthogonalised.
cudaError_t launch_ortho_norms(const OrthoPrep& p, cudaStream_t stream);
// X = u / (|u| + eps) as planes.
cudaError_t launch_ortho_planes(const OrthoPrep& p, cudaStream_t stream);

}  // namespace ddl
