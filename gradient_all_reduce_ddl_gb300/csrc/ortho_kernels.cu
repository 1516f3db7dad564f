// ortho_kernels.cu -- what comes before the Newton-Schulz products: the momentum
// step, the matrices' Frobenius norms and the first iterate's planes.  Both
// kernels are bound by HBM (or L2) traffic.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ortho_kernels.h"
#include "product.h"

namespace ddl {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load_elem(const void* base, int64_t at, int type) {
  if (type == kF32) return static_cast<const float*>(base)[at];
  const uint16_t u = static_cast<const uint16_t*>(base)[at];
  return type == kBF16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}

// Place of row-major element e.
__device__ __forceinline__ void locate(const OrthoMatrix& m, int64_t e, int64_t* flat, int64_t* plane) {
  int64_t r;
  if (m.rows * m.cols < (1ll << 31))
    r = (uint32_t)e / (uint32_t)m.cols;
  else
    r = e / m.cols;
  const int64_t c = e - r * m.cols;
  *flat = m.offset + r * m.ld + c;
  *plane = r * m.ldp + c;
}

// The sum over the CTA's threads, in a fixed order, for thread 0.
__device__ __forceinline__ double block_sum(double s) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_down_sync(0xffffffffu, s, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < kThreads / 32; ++w) s += part[w];
  return s;
}

__global__ void __launch_bounds__(kThreads) norms_kernel(const OrthoPrep p) {
  const OrthoItem it = p.items[blockIdx.x];
  const OrthoMatrix m = p.matrices[it.matrix];
  double s = 0;
  for (int64_t e = it.begin + threadIdx.x; e < it.end; e += kThreads) {
    int64_t at, plane;
    locate(m, e, &at, &plane);
    float u = load_elem(p.in, at, p.type);
    if (p.mom) {
      const float g = u, v = p.mu * p.mom[at] + g;
      p.mom[at] = v;
      u = p.nesterov ? g + p.mu * v : v;
    }
    s += (double)u * (double)u;  // binary64: squares of any binary32 value are in range
  }
  s = block_sum(s);
  if (threadIdx.x == 0) p.partial[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) planes_kernel(const OrthoPrep p) {
  __shared__ float inv;
  const OrthoItem it = p.items[blockIdx.x];
  const OrthoMatrix m = p.matrices[it.matrix];
  double s = 0;
  for (int i = threadIdx.x; i < m.n_items; i += kThreads) s += p.partial[m.item0 + i];
  s = block_sum(s);
  if (threadIdx.x == 0) inv = (float)(1.0 / (sqrt(s) + (double)p.eps));
  __syncthreads();
  const float scale = inv;
  for (int64_t e = it.begin + threadIdx.x; e < it.end; e += kThreads) {
    int64_t at, plane;
    locate(m, e, &at, &plane);
    float u = load_elem(p.in, at, p.type);
    if (p.mom) {
      const float g = u, v = p.mom[at];
      u = p.nesterov ? g + p.mu * v : v;
    }
    const float x = u * scale;
    const __half h = __float2half_rn(x);
    const float hf = __half2float(h);
    m.hi[plane] = __half_as_ushort(h);
    m.lo[plane] = isfinite(hf) ? __half_as_ushort(__float2half_rn((x - hf) * 2048.f)) : (uint16_t)0;
  }
}

}  // namespace

cudaError_t launch_ortho_norms(const OrthoPrep& p, cudaStream_t stream) {
  norms_kernel<<<(unsigned)p.n_items, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_ortho_planes(const OrthoPrep& p, cudaStream_t stream) {
  planes_kernel<<<(unsigned)p.n_items, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace ddl
