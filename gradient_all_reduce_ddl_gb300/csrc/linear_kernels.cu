// linear_kernels.cu -- the launch before a linear layer's products: dz = dy act'(z)
// as 16-bit planes, its column sums (the bias gradient), and copies of operands
// whose rows are not 16-byte aligned.  One launch for all of it: small layers are
// bound by launches (256 x 1000 column sums: 4.6 us).  Large ones are bound by HBM traffic
// (with binary32 gradients a bfloat16 dz reads 4 and writes 6 bytes an element: 8192 x
// 8192 with GELU 127 us, 5.3 TB/s of 6.8) and by the slope's arithmetic.
#include "activation.cuh"
#include "linear_kernels.h"
#include "product.h"
#include "tc_ptx.cuh"

namespace ddl {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPackRows = 32, kPackCols = 256;  // what a CTA copies

__device__ __forceinline__ void pack_block(const Pack& p, int64_t block) {
  const int64_t across = (p.cols + kPackCols - 1) / kPackCols;
  const int64_t row0 = block / across * kPackRows + (threadIdx.x >> 5), col0 = block % across * kPackCols + (threadIdx.x & 31);
#pragma unroll
  for (int i = 0; i < kPackRows / kWarps; ++i) {
    const int64_t r = row0 + i * kWarps;
    if (r >= p.rows) break;
    uint16_t v[kPackCols / 32];
#pragma unroll
    for (int j = 0; j < kPackCols / 32; ++j)
      if (col0 + 32 * j < p.cols) v[j] = p.src[r * p.ld + col0 + 32 * j];
#pragma unroll
    for (int j = 0; j < kPackCols / 32; ++j)
      if (col0 + 32 * j < p.cols) p.dst[r * p.ldp + col0 + 32 * j] = v[j];
  }
}

// The planes of two neighbours.  One plane: the values in the operand's type (exact for no activation and ReLU).
// bfloat16: up to three 8-bit parts.  binary16: half the value (so that a slope above one cannot overflow), and 2^11
// times what its rounding lost.  Infinities and NaNs stay in the first plane alone.
template <int TYPE, int N>
__device__ __forceinline__ void planes_of(float x, float y, uint32_t (&out)[kMaxPlanes]) {
  if constexpr (TYPE == kBF16 || N == 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      out[k] = to16x2(x, y, TYPE);
      const float2 h = from16x2(out[k], TYPE);
      // an infinite or NaN part leaves nothing for the next one
      x = isfinite(h.x) ? x - h.x : 0.f;
      y = isfinite(h.y) ? y - h.y : 0.f;
    }
  } else {
    x *= 0.5f, y *= 0.5f;
    out[0] = to16x2(x, y, kF16);
    const float2 h = from16x2(out[0], kF16);
    out[1] = to16x2(isfinite(h.x) ? (x - h.x) * 2048.f : 0.f, isfinite(h.y) ? (y - h.y) * 2048.f : 0.f, kF16);
  }
}

// block_rows x kDzCols of dz; warp w has the rows w, w + 8, ..., a lane 8 columns: neighbours (VEC) or 32 apart.
template <int TYPE, int ACT, int N, bool VEC>
__device__ __forceinline__ void dz_rows(const LinearPrep& p, int64_t r0, int64_t c0, float (&sum)[8]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint16_t* dy = static_cast<const uint16_t*>(p.dy);
  const uint16_t* zp = static_cast<const uint16_t*>(p.z);
  if (VEC && c0 + 8 * lane >= p.cols) return;
#pragma unroll 2
  for (int i = warp; i < p.block_rows; i += kWarps) {
    const int64_t r = r0 + i;
    if (r >= p.rows) break;
    float v[8], z[8];
    if constexpr (VEC) {
      const int64_t c = c0 + 8 * lane;
      const uint4 g = *reinterpret_cast<const uint4*>(dy + r * p.ldy + c);
      uint4 u = make_uint4(0, 0, 0, 0);
      if (ACT != kActNone) u = *reinterpret_cast<const uint4*>(zp + r * p.ldz + c);
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, zw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = from16x2(gw[j], TYPE), b = from16x2(zw[j], TYPE);
        v[2 * j] = a.x, v[2 * j + 1] = a.y, z[2 * j] = b.x, z[2 * j + 1] = b.y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t c = c0 + lane + 32 * j;
        v[j] = c < p.cols ? from16(dy[r * p.ldy + c], TYPE) : 0.f;
        z[j] = ACT != kActNone && c < p.cols ? from16(zp[r * p.ldz + c], TYPE) : 0.f;
      }
    }
    uint32_t out[4][kMaxPlanes];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (ACT == kActRelu) {  // a closed unit passes nothing on, whatever dy is
        v[2 * j] = z[2 * j] > 0.f ? v[2 * j] : 0.f;
        v[2 * j + 1] = z[2 * j + 1] > 0.f ? v[2 * j + 1] : 0.f;
      } else if (ACT != kActNone) {
        v[2 * j] *= act_slope(z[2 * j], ACT);
        v[2 * j + 1] *= act_slope(z[2 * j + 1], ACT);
      }
      sum[2 * j] += v[2 * j];
      sum[2 * j + 1] += v[2 * j + 1];
      if constexpr (N > 0) planes_of<TYPE, N>(v[2 * j], v[2 * j + 1], out[j]);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if constexpr (VEC) {
        *reinterpret_cast<uint4*>(p.planes[k] + r * p.ldp + c0 + 8 * lane) =
            make_uint4(out[0][k], out[1][k], out[2][k], out[3][k]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t c = c0 + lane + 32 * j;
          if (c < p.cols) p.planes[k][r * p.ldp + c] = (uint16_t)(out[j >> 1][k] >> (j & 1) * 16);
        }
      }
    }
  }
}

template <int TYPE, int ACT, bool VEC>
__device__ __forceinline__ void dz_planes(const LinearPrep& p, int64_t r0, int64_t c0, float (&sum)[8]) {
  // GELU and SiLU take as many planes as the results ask for, up to three of bfloat16; the others one, or none
  constexpr bool kCurved = ACT == kActGelu || ACT == kActSilu;
  constexpr int kTwo = kCurved ? 2 : 1, kMost = kCurved && TYPE == kBF16 ? 3 : kTwo;
  if (p.n_planes == 0)
    dz_rows<TYPE, ACT, 0, VEC>(p, r0, c0, sum);
  else if (p.n_planes == 1)
    dz_rows<TYPE, ACT, 1, VEC>(p, r0, c0, sum);
  else if (p.n_planes == 2)
    dz_rows<TYPE, ACT, kTwo, VEC>(p, r0, c0, sum);
  else
    dz_rows<TYPE, ACT, kMost, VEC>(p, r0, c0, sum);
}

template <int TYPE, bool VEC>
__device__ __forceinline__ void dz_act(const LinearPrep& p, int64_t r0, int64_t c0, float (&sum)[8]) {
  switch (p.z ? p.act : kActNone) {
    case kActRelu: dz_planes<TYPE, kActRelu, VEC>(p, r0, c0, sum); break;
    case kActGelu: dz_planes<TYPE, kActGelu, VEC>(p, r0, c0, sum); break;
    case kActSilu: dz_planes<TYPE, kActSilu, VEC>(p, r0, c0, sum); break;
    default: dz_planes<TYPE, kActNone, VEC>(p, r0, c0, sum); break;
  }
}

template <int TYPE, bool VEC>
__global__ void __launch_bounds__(kThreads) prep_kernel(const __grid_constant__ LinearPrep p) {
  __shared__ float sums[kWarps][kDzCols];
  __shared__ bool last;
  tc::griddep_launch();
  tc::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t across = (p.cols + kDzCols - 1) / kDzCols, down = (p.rows + p.block_rows - 1) / p.block_rows;
  int64_t block = blockIdx.x;
  const int64_t dz_blocks = p.has_dz ? across * down : 0;
  if (block >= dz_blocks) {
    block -= dz_blocks;
    const int64_t first = (p.pack[0].rows + kPackRows - 1) / kPackRows * ((p.pack[0].cols + kPackCols - 1) / kPackCols);
    if (block < first)
      pack_block(p.pack[0], block);
    else
      pack_block(p.pack[1], block - first);
    return;
  }
  const int64_t cb = block / down, rb = block % down, c0 = cb * kDzCols;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  dz_act<TYPE, VEC>(p, rb * p.block_rows, c0, sum);
  if (!p.db) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[warp][VEC ? 8 * lane + j : lane + 32 * j] = sum[j];
  __syncthreads();
  const int64_t c = c0 + threadIdx.x;
  if (c < p.cols) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w][threadIdx.x];
    p.partial[rb * p.cols + c] = s;
  }
  // the last CTA of these columns adds the row blocks' sums: a warp every eighth of them, then the warps, always in this
  // order
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(p.done + cb, 1u) == (uint32_t)(down - 1);
  __syncthreads();
  if (!last) return;
  __threadfence();
  if (threadIdx.x == 0) p.done[cb] = 0;  // for the next call
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = 0.f;
#pragma unroll 2
  for (int64_t b = warp; b < down; b += kWarps) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t at = c0 + lane + 32 * j;
      sum[j] += at < p.cols ? __ldcg(p.partial + b * p.cols + at) : 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[warp][lane + 32 * j] = sum[j];
  __syncthreads();
  if (c >= p.cols) return;
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += sums[w][threadIdx.x];
  if (p.db_f32) {
    float* o = static_cast<float*>(p.db) + c;
    *o = p.accumulate ? *o + s : s;
  } else {
    __half* o = static_cast<__half*>(p.db) + c;
    *o = __float2half_rn(p.accumulate ? __half2float(*o) + s : s);
  }
}

}  // namespace

float plane_scale(int type, int n, int k) {
  if (type == kBF16 || n == 1) return 1.f;
  return k == 0 ? 2.f : 2.f / 2048.f;
}

cudaError_t launch_linear_prep(const LinearPrep& p, cudaStream_t stream) {
  int64_t blocks = p.has_dz ? ((p.cols + kDzCols - 1) / kDzCols) * ((p.rows + p.block_rows - 1) / p.block_rows) : 0;
  for (int k = 0; k < p.n_packs; ++k)
    blocks += ((p.pack[k].rows + kPackRows - 1) / kPackRows) * ((p.pack[k].cols + kPackCols - 1) / kPackCols);
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const auto kernel = p.type == kBF16 ? (p.vec ? prep_kernel<kBF16, true> : prep_kernel<kBF16, false>)
                                      : (p.vec ? prep_kernel<kF16, true> : prep_kernel<kF16, false>);
  return tc::launch_early(kernel, dim3((unsigned)blocks), kThreads, stream, p);
}

}  // namespace ddl
