// layer_util.h -- what the C entry points of the linear layers and of the loss share: workspaces, the caller's matrices and
// their checks, tensor maps (internal).
#pragma once

#include <algorithm>
#include <cstdint>

#include "api_util.h"
#include "ddl.h"
#include "linear_kernels.h"
#include "product.h"

namespace ddl {

// K blocks that stay in the tensor core's truncating accumulator for 16-bit results.  Each of a block's four additions
// loses up to half a unit in the last place of the partial sum, 2^-24 of it: 256 blocks 2^-14 of a sum of one sign, a quarter
// of binary16's half unit (2^-12 at least), 2048 blocks a quarter of bfloat16's.
inline int64_t long_chunk(int type) { return type == kF16 ? 256 : 2048; }
// K blocks of a binary32 result: what the truncating accumulator loses of a chunk does not average out, while a sum in
// binary32 loses less the shorter it is.  With these chunks dw's error over the sizes measured (64 to 65,536 tokens,
// normal inputs, dz exact) is 0.2 to 1.34 times that of products in binary32; with 8 blocks throughout it was up to 5.4
// times, with 4 up to 2.7.  A sum of one sign ends 0.8, 1.5 and 3.1e-7 off with 1, 2 and 4 blocks.  Against 8 blocks they
// cost 5 to 9 % of a call of 512 to 2048 tokens (512, 2048 -> 4096 with GELU 64.9 -> 69.4 us; a square layer of 2048
// without 37.2 -> 41.1) and 2 to 5 % of 8192 (2048 -> 8192: 941 -> 957 and 398 -> 417 us).
inline int32_t f32_chunk(int64_t tokens) { return tokens <= 640 ? 1 : tokens <= 2048 ? 2 : 4; }

struct Buffer {  // device memory that grows with the first calls that need it
  void* p = nullptr;
  size_t bytes = 0;
};

inline ddl_status_t need(Buffer* b, size_t bytes) {
  if (b->bytes >= bytes) return DDL_OK;
  void* p = nullptr;
  const cudaError_t e = device_alloc(&p, bytes);
  if (e != cudaSuccess) return status_of(e);
  // never outgrown: the sizes asked for are the handle's maxima
  b->p = p;
  b->bytes = bytes;
  return DDL_OK;
}

// A rows x cols 16-bit matrix as the caller gave it.
struct Mat {
  const void* p;
  int64_t rows, cols, ld;
  Range range(int esize) const {
    return Range(p, p && rows ? ((uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)cols) * (uint64_t)esize : 0);
  }
  bool tma() const { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; }
  bool tma32() const { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 4 == 0; }
  bool vec4(int esize) const { return reinterpret_cast<uintptr_t>(p) % (4 * (size_t)esize) == 0 && ld % 4 == 0; }
};

inline bool fits(int64_t rows, int64_t ld, int64_t cols) {
  return ld >= cols && ld <= (1ll << 31) && rows <= (1ll << 60) / ld;
}

// The matrix itself, or where the preparing launch copies it with 16-byte aligned rows.
inline ddl_status_t aligned(const Mat& m, int64_t max_rows, Buffer* b, LinearPrep* prep, Mat* out) {
  *out = m;
  if (m.tma()) return DDL_OK;
  const int64_t ldp = (int64_t)round8((uint64_t)m.cols);
  const ddl_status_t st = need(b, (size_t)max_rows * (size_t)ldp * 2);
  if (st != DDL_OK) return st;
  *out = Mat{b->p, m.rows, m.cols, ldp};
  prep->pack[prep->n_packs++] = {static_cast<const uint16_t*>(m.p), m.ld, static_cast<uint16_t*>(b->p), ldp, m.rows, m.cols};
  return DDL_OK;
}

inline bool map_of(ProductLaunch* L, int k, const Mat& m, int box_cols, int box_rows = 0) {
  if (!box_rows) box_rows = box_cols == kSlabCols ? kTileM : kBoxRows;
  return make_map(&L->maps[k], m.p, (uint64_t)m.rows, (uint64_t)m.cols, (uint64_t)m.ld, box_cols, box_rows,
                  L->bf16 != 0);
}

inline bool map32_of(ProductLaunch* L, int k, const Mat& m) {
  return make_map32(&L->maps[k], m.p, (uint64_t)m.rows, (uint64_t)m.cols, (uint64_t)m.ld);
}

inline int64_t blocks_of(int64_t n, int64_t b) { return (n + b - 1) / b; }

// Whether two matrices (element sizes ea, eb) have a byte in common.  Matrices of one row pitch may interleave: column
// blocks of the same wider buffer.
inline bool overlap(const Mat& a, int ea, const Mat& b, int eb) {
  if (!a.range(ea).overlaps(b.range(eb))) return false;
  const uint64_t pitch = (uint64_t)a.ld * (uint64_t)ea;
  if (pitch != (uint64_t)b.ld * (uint64_t)eb) return true;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const uint64_t off = pb >= pa ? (pb - pa) % pitch : (pitch - (pa - pb) % pitch) % pitch;  // b's columns in a's rows
  return off < (uint64_t)a.cols * (uint64_t)ea || off + (uint64_t)b.cols * (uint64_t)eb > pitch;
}

struct Operand {
  Mat m;
  int esize;
};

// Nothing written meets anything else, and no range wraps around.
inline bool distinct(const Operand* out, int n_out, const Operand* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    if (out[i].m.range(out[i].esize).wraps()) return false;
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(out[i].m, out[i].esize, out[j].m, out[j].esize)) return false;
    for (int j = 0; j < n_in; ++j)
      if (in[j].m.range(in[j].esize).wraps() || overlap(out[i].m, out[i].esize, in[j].m, in[j].esize)) return false;
  }
  return true;
}

}  // namespace ddl
