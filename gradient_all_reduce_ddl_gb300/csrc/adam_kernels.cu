// adam_kernels.cu -- the AdamW step over many tensors of a flat buffer, on every
// worker's copy of the parameters, and the gradient's norm.
//
//   g' = c g;   m = b1 m + (1 - b1) g';   v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Bound by HBM: 28 bytes an element with binary32 states and one copy, 8 (10 with a
// 16-bit operand copy) for each further copy.  One launch covers every tensor: a warp
// takes an item of up to 1024 elements of one tensor, a block of 128 at a time, four
// elements per lane, so that a block's largest value (the 8-bit states' scale) is one
// warp reduction and the work does not depend on how long the tensors are.
//
// Products and sums are rounded one by one (no fused multiply-adds), as in the fused
// SGD update, so that the states are the same bits as in a step-by-step evaluation.
#include <cuda_fp8.h>

#include "activation.cuh"
#include "adam_kernels.h"
#include "tc_ptx.cuh"

namespace ddl {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr float kTop = 448.f;             // e4m3's largest number
constexpr float kLeast = 0x1p-100f;       // blocks whose largest value is below this are kept as zeros
constexpr uint8_t kCodeNan = 0x7F;

// Element j of a lane: neighbours (V = 4), or 32 apart (V = 1: any alignment, and a tensor's last block).
template <int V>
__device__ __forceinline__ uint32_t place(int lane, int j) {
  return V == 4 ? 4 * lane + j : lane + 32 * j;
}

template <int V>
__device__ __forceinline__ void load32(const float* p, uint32_t len, int lane, float (&x)[4]) {
  if constexpr (V == 4) {
    const float4 u = *reinterpret_cast<const float4*>(p + 4 * lane);
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = place<V>(lane, j) < len ? p[place<V>(lane, j)] : 0.f;
  }
}

template <int V>
__device__ __forceinline__ void store32(float* p, uint32_t len, int lane, const float (&x)[4]) {
  if constexpr (V == 4) {
    *reinterpret_cast<float4*>(p + 4 * lane) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (place<V>(lane, j) < len) p[place<V>(lane, j)] = x[j];
  }
}

template <int V>
__device__ __forceinline__ void load_grad(const void* base, int64_t at, int type, uint32_t len, int lane, float (&x)[4]) {
  if (type == kF32) {
    load32<V>(static_cast<const float*>(base) + at, len, lane, x);
    return;
  }
  const uint16_t* p = static_cast<const uint16_t*>(base) + at;
  if constexpr (V == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p + 4 * lane);
    const float2 a = from16x2(u.x, kF16), b = from16x2(u.y, kF16);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = place<V>(lane, j) < len ? from16(p[place<V>(lane, j)], kF16) : 0.f;
  }
}

template <int V>
__device__ __forceinline__ void store16(void* base, int64_t at, int type, uint32_t len, int lane, const float (&x)[4]) {
  uint16_t* p = static_cast<uint16_t*>(base) + at;
  if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(p + 4 * lane) = make_uint2(to16x2(x[0], x[1], type), to16x2(x[2], x[3], type));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (place<V>(lane, j) < len) p[place<V>(lane, j)] = to16(x[j], type);
  }
}

// -- 8-bit states -----------------------------------------------------------------
//
// A block's values are e4m3 codes of value x (448 / largest) and the scale largest / 448.  e4m3 keeps 4 bits of values
// down to 2^-15 of the largest and goes on to 2^-18; of v the square root is kept, whose range is half as wide, and a
// root that is not zero never becomes zero, since the step divides by it.  An infinite or NaN value is a NaN code and
// does not touch the block's others.

template <int V>
__device__ __forceinline__ void load_codes(const void* base, int64_t at, uint32_t len, int lane, float scale, float (&x)[4]) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + at;
  uint32_t u = 0;
  if constexpr (V == 4) {
    u = *reinterpret_cast<const uint32_t*>(p + 4 * lane);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (place<V>(lane, j) < len) u |= (uint32_t)p[place<V>(lane, j)] << (8 * j);
  }
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u & 0xFFFFu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> 16), __NV_E4M3);
  const float2 f = __half22float2(__half2(a)), g = __half22float2(__half2(b));
  x[0] = f.x * scale, x[1] = f.y * scale, x[2] = g.x * scale, x[3] = g.y * scale;
}

// Encodes a block's values (zeros outside the tensor) and returns its scale.
template <int V, bool ROOT>
__device__ __forceinline__ float store_codes(void* base, int64_t at, uint32_t len, int lane, const float (&x)[4]) {
  uint32_t most = 0;  // largest finite magnitude: as bits they order as the numbers do
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t b = __float_as_uint(x[j]) & 0x7FFFFFFFu;
    most = b < 0x7F800000u && b > most ? b : most;
  }
  const float top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, most));
  const bool held = top >= kLeast;
  const float by = held ? kTop / top : 0.f;
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * by, x[1] * by), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * by, x[3] * by), __NV_SATFINITE, __NV_E4M3);
  uint32_t u = (uint32_t)lo | (uint32_t)hi << 16;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t mask = 0xFFu << (8 * j);
    if (ROOT && held && x[j] > 0.f && !(u & mask)) u |= 1u << (8 * j);
    if (!(fabsf(x[j]) < INFINITY)) u = (u & ~mask) | (uint32_t)kCodeNan << (8 * j);
  }
  uint8_t* p = static_cast<uint8_t*>(base) + at;
  if constexpr (V == 4) {
    *reinterpret_cast<uint32_t*>(p + 4 * lane) = u;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (place<V>(lane, j) < len) p[place<V>(lane, j)] = (uint8_t)(u >> (8 * j));
  }
  return held ? top / kTop : 0.f;
}

// -- the step -----------------------------------------------------------------------

// What the step count and the norm make of the parameters, in every thread.
struct Factors {
  float scale;  // of the gradient
  float size;   // lr / (1 - b1^t)
  float root;   // sqrt(1 - b2^t)
};

template <int BITS, int V>
__device__ __forceinline__ void block_step(const AdamStep& p, const Factors& f, const AdamItem& it, uint32_t first,
                                           uint32_t len, int lane) {
  const int64_t at = (int64_t)(it.begin + first);
  const uint32_t block = it.block + first / kAdamBlock;
  float g[4], m[4], v[4], t[4][4];
  load_grad<V>(p.grad, at, p.grad_type, len, lane, g);
  if constexpr (BITS == 32) {
    load32<V>(static_cast<const float*>(p.m) + at, len, lane, m);
    load32<V>(static_cast<const float*>(p.v) + at, len, lane, v);
  } else {
    load_codes<V>(p.m, at, len, lane, p.scale_m[block], m);
    load_codes<V>(p.v, at, len, lane, p.scale_v[block], v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= v[j];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < p.n_copies) load32<V>(p.params[k] + at, len, lane, t[k]);
  const float size = f.size * it.lr, keep = 1.f - p.lr * it.lr * p.weight_decay * it.decay;
  float u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    g[j] *= f.scale;
    m[j] = m[j] * p.beta1 + g[j] * p.rest1;
    v[j] = v[j] * p.beta2 + g[j] * p.rest2 * g[j];
    const float root = sqrtf(v[j]);
    u[j] = m[j] / (root / f.root + p.eps) * size;
    if (BITS == 8) v[j] = root;
  }
  if constexpr (BITS == 32) {
    store32<V>(static_cast<float*>(p.m) + at, len, lane, m);
    store32<V>(static_cast<float*>(p.v) + at, len, lane, v);
  } else {
    const float sm = store_codes<V, false>(p.m, at, len, lane, m), sv = store_codes<V, true>(p.v, at, len, lane, v);
    if (lane == 0) p.scale_m[block] = sm, p.scale_v[block] = sv;
  }
#pragma unroll 1
  for (int c = 0; c < p.n_copies; c += 4) {
    if (c > 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c + k < p.n_copies) load32<V>(p.params[c + k] + at, len, lane, t[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (c + k >= p.n_copies) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) t[k][j] = t[k][j] * keep - u[j];
      store32<V>(p.params[c + k] + at, len, lane, t[k]);
      if (p.out[0]) store16<V>(p.out[c + k], at, p.out_type, len, lane, t[k]);
    }
  }
}

template <int BITS>
__global__ void __launch_bounds__(kThreads) step_kernel(const __grid_constant__ AdamStep p) {
  const int lane = threadIdx.x & 31;
  tc::griddep_launch();
  tc::griddep_wait();
  const int64_t t = *p.step + 1;
  Factors f;
  // 1 - b^t = -expm1(t log b): the difference would lose what is left of a beta near one
  f.size = p.lr / -expm1f((float)((double)t * p.log_beta1));
  f.root = sqrtf(-expm1f((float)((double)t * p.log_beta2)));
  f.scale = p.norm ? p.norm->scale : p.grad_scale;
  for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < p.n_items; i += (int64_t)gridDim.x * kWarps) {
    const AdamItem it = p.items[i];
    const bool vec = p.vec && it.begin % 4 == 0;
#pragma unroll 1
    for (uint32_t first = 0; first < it.len; first += kAdamBlock) {
      const uint32_t len = it.len - first < kAdamBlock ? it.len - first : kAdamBlock;
      if (vec && len == kAdamBlock)
        block_step<BITS, 4>(p, f, it, first, len, lane);
      else
        block_step<BITS, 1>(p, f, it, first, len, lane);
    }
  }
  // the last CTA counts the step: every other one has read the count
  __syncthreads();
  if (threadIdx.x == 0 && atomicInc(p.done, gridDim.x - 1) == gridDim.x - 1) *p.step = t;
}

// -- the gradient's norm ---------------------------------------------------------------

template <int V>
__device__ __forceinline__ double block_squares(const AdamStep& p, int64_t at, uint32_t len, int lane) {
  float g[4];
  load_grad<V>(p.grad, at, p.grad_type, len, lane, g);
  const float s = (g[0] * g[0] + g[1] * g[1]) + (g[2] * g[2] + g[3] * g[3]);
  // squares that leave binary32's range are taken again in 64 bits
  if (s > 0x1p-80f && s < 0x1p100f) return (double)s;
  double d = 0.0;
  if (g[0] != 0.f || g[1] != 0.f || g[2] != 0.f || g[3] != 0.f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) d += (double)g[j] * (double)g[j];
  }
  return d;
}

__device__ __forceinline__ double block_sum(double v, double* shared) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_down_sync(0xFFFFFFFFu, v, d);
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kWarps; ++w) v += shared[w];
  return v;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ AdamStep p) {
  __shared__ double sums[2][kWarps];
  __shared__ bool last;
  const int lane = threadIdx.x & 31;
  tc::griddep_launch();
  tc::griddep_wait();
  double s = 0.0;
  for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < p.n_items; i += (int64_t)gridDim.x * kWarps) {
    const AdamItem it = p.items[i];
    const bool vec = p.vec && it.begin % 4 == 0;
#pragma unroll 4
    for (uint32_t first = 0; first < it.len; first += kAdamBlock) {
      const uint32_t len = it.len - first < kAdamBlock ? it.len - first : kAdamBlock;
      const int64_t at = (int64_t)(it.begin + first);
      s += vec && len == kAdamBlock ? block_squares<4>(p, at, len, lane) : block_squares<1>(p, at, len, lane);
    }
  }
  s = block_sum(s, sums[0]);
  if (threadIdx.x == 0) {
    p.norm->parts[blockIdx.x] = s;
    __threadfence();
    last = atomicInc(p.done + 1, gridDim.x - 1) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  // the CTAs' sums, always in the same order
  s = 0.0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kThreads) s += __ldcg(p.norm->parts + i);
  s = block_sum(s, sums[1]);
  if (threadIdx.x == 0) {
    const float norm = (float)(sqrt(s) * fabs((double)p.grad_scale));
    if (p.norm_out) *p.norm_out = norm;
    float scale = p.grad_scale;
    if (p.max_norm > 0.f) {
      const float by = p.max_norm / (norm + 1e-6f);
      if (!(by >= 1.f)) scale *= by;  // a NaN stays one
    }
    p.norm->scale = scale;
  }
}

unsigned grid_of(const AdamStep& p, int sms, int most) {
  const int64_t ctas = (p.n_items + kWarps - 1) / kWarps, wave = (int64_t)sms * most;
  return (unsigned)(ctas < wave ? ctas : wave);
}

}  // namespace

cudaError_t launch_adam_norm(const AdamStep& p, int sms, cudaStream_t stream) {
  unsigned grid = grid_of(p, sms, 8);
  if (grid > kMaxNormParts) grid = kMaxNormParts;
  return tc::launch_early(norm_kernel, dim3(grid), kThreads, stream, p);
}

cudaError_t launch_adam_step(const AdamStep& p, int sms, cudaStream_t stream) {
  return p.bits == 8 ? tc::launch_early(step_kernel<8>, dim3(grid_of(p, sms, 8)), kThreads, stream, p)
                     : tc::launch_early(step_kernel<32>, dim3(grid_of(p, sms, 8)), kThreads, stream, p);
}

}  // namespace ddl
