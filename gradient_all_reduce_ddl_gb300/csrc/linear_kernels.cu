// linear_kernels.cu -- the linear layers' element-wise kernels: dz = dy act'(z)
// as 16-bit planes with its column sums (the bias gradient), and the copy of
// matrices whose rows are not 16-byte aligned.  All are bound by HBM traffic.
#include "activation.cuh"
#include "linear_kernels.h"
#include "product.h"
#include "tc_ptx.cuh"

namespace ddl {
namespace {

__global__ void pack16_kernel(const uint16_t* __restrict__ src, int64_t ld, uint16_t* __restrict__ dst, int64_t ldp,
                              int64_t rows, int64_t cols) {
  tc::griddep_launch();
  tc::griddep_wait();
  const int64_t col0 = (int64_t)blockIdx.x * 256 + (threadIdx.x & 31);
  for (int64_t r = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5); r < rows; r += (int64_t)gridDim.y * 8) {
    uint16_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col0 + 32 * j < cols) v[j] = src[r * ld + col0 + 32 * j];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col0 + 32 * j < cols) dst[r * ldp + col0 + 32 * j] = v[j];
  }
}

// The planes of one value.  One plane: the value in the operand's type (exact
// for no activation and ReLU).  bfloat16: up to three 8-bit parts.  binary16: half
// the value (so that a slope above one cannot overflow), and 2^11 times what its
// rounding lost.  Infinities and NaNs stay in the first plane alone.
__device__ __forceinline__ void planes_of(float v, int type, int n, uint16_t (&out)[kMaxPlanes]) {
  out[1] = out[2] = 0;
  if (type == kBF16) {
    float r = v;
#pragma unroll
    for (int k = 0; k < kMaxPlanes; ++k) {
      if (k >= n) break;
      const __nv_bfloat16 h = __float2bfloat16_rn(r);
      out[k] = __bfloat16_as_ushort(h);
      const float hf = __bfloat162float(h);
      if (!isfinite(hf)) break;
      r -= hf;
    }
  } else if (n == 1) {
    out[0] = __half_as_ushort(__float2half_rn(v));
  } else {
    const float x = 0.5f * v;
    const __half h = __float2half_rn(x);
    const float hf = __half2float(h);
    out[0] = __half_as_ushort(h);
    if (isfinite(hf)) out[1] = __half_as_ushort(__float2half_rn((x - hf) * 2048.f));
  }
}

// A CTA takes 128 columns x kDzRows rows; warp w the rows w, w + 8, ...
template <bool VEC>
__global__ void __launch_bounds__(256) dz_kernel(const DzParams p) {
  tc::griddep_launch();
  tc::griddep_wait();
  __shared__ float sums[8][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c0 = (int64_t)blockIdx.y * 128, r0 = (int64_t)blockIdx.x * kDzRows;
  const uint16_t* dy = static_cast<const uint16_t*>(p.dy);
  const uint16_t* zp = static_cast<const uint16_t*>(p.z);
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int i = warp; i < kDzRows; i += 8) {
    const int64_t r = r0 + i;
    if (r >= p.rows) break;
    uint16_t g[4], z[4];
    uint16_t out[4][kMaxPlanes];
    if constexpr (VEC) {
      const int64_t c = c0 + 4 * lane;
      if (c >= p.cols) continue;
      *reinterpret_cast<ushort4*>(g) = *reinterpret_cast<const ushort4*>(dy + r * p.ldy + c);
      if (zp) *reinterpret_cast<ushort4*>(z) = *reinterpret_cast<const ushort4*>(zp + r * p.ldz + c);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t c = c0 + lane + 32 * j;
        g[j] = c < p.cols ? dy[r * p.ldy + c] : (uint16_t)0;
        z[j] = zp && c < p.cols ? zp[r * p.ldz + c] : (uint16_t)0;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v = from16(g[j], p.type);
      if (zp) v *= act_slope(from16(z[j], p.type), p.act);
      sum[j] += v;
      if (p.n_planes) planes_of(v, p.type, p.n_planes, out[j]);
    }
#pragma unroll
    for (int k = 0; k < kMaxPlanes; ++k) {
      if (k >= p.n_planes) break;
      if constexpr (VEC) {
        *reinterpret_cast<ushort4*>(p.planes[k] + r * p.ldp + c0 + 4 * lane) =
            make_ushort4(out[0][k], out[1][k], out[2][k], out[3][k]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c0 + lane + 32 * j < p.cols) p.planes[k][r * p.ldp + c0 + lane + 32 * j] = out[j][k];
      }
    }
  }
  if (!p.partial) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) sums[warp][VEC ? 4 * lane + j : lane + 32 * j] = sum[j];
  __syncthreads();
  if (threadIdx.x < 128 && c0 + threadIdx.x < p.cols) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sums[w][threadIdx.x];
    p.partial[(int64_t)blockIdx.x * p.cols + c0 + threadIdx.x] = s;
  }
}

// 32 columns a CTA; warp w adds the row blocks w, w + 8, ..., then the warps' sums are added in order.
__global__ void __launch_bounds__(256) db_kernel(const float* __restrict__ partial, int64_t blocks, int64_t cols,
                                                 void* db, int type, int accumulate) {
  tc::griddep_launch();
  tc::griddep_wait();
  __shared__ float sums[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols)
    for (int64_t b = warp; b < blocks; b += 8) s += partial[b * cols + c];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= cols) return;
#pragma unroll
  for (int w = 1; w < 8; ++w) s += sums[w][lane];
  if (type == kF32) {
    float* o = static_cast<float*>(db) + c;
    *o = accumulate ? *o + s : s;
  } else {
    __half* o = static_cast<__half*>(db) + c;
    *o = __float2half_rn(accumulate ? __half2float(*o) + s : s);
  }
}

}  // namespace

float plane_scale(int type, int n, int k) {
  if (type == kBF16 || n == 1) return 1.f;
  return k == 0 ? 2.f : 2.f / 2048.f;
}

cudaError_t launch_pack16(const void* src, int64_t ld, void* dst, int64_t ldp, int64_t rows, int64_t cols,
                          cudaStream_t stream) {
  const int64_t by = (rows + 7) / 8;
  const dim3 grid((unsigned)((cols + 255) / 256), (unsigned)(by < 65535 ? by : 65535));
  return tc::launch_early(pack16_kernel, grid, 256, stream, static_cast<const uint16_t*>(src), ld,
                          static_cast<uint16_t*>(dst), ldp, rows, cols);
}

cudaError_t launch_dz(const DzParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.rows + kDzRows - 1) / kDzRows), (unsigned)((p.cols + 127) / 128));
  return tc::launch_early(p.vec ? dz_kernel<true> : dz_kernel<false>, grid, 256, stream, p);
}

cudaError_t launch_db(const float* partial, int64_t blocks, int64_t cols, void* db, int type, int accumulate,
                      cudaStream_t stream) {
  return tc::launch_early(db_kernel, dim3((unsigned)((cols + 31) / 32)), 256, stream, partial, blocks, cols, db, type,
                          accumulate);
}

}  // namespace ddl
