// ortho_kernels.cu -- what comes before and after the Newton-Schulz products: the
// momentum step, the matrices' Frobenius norms and the first iterate's planes;
// the result or the parameter step from the last iterate's planes.
//
// All are bound by HBM (or L2) traffic.  A CTA takes an item of 1024 to 8192
// elements, four to a thread at a time where the layout allows it, with the
// loads of four such groups issued together (the parameter step: of four copies).
// The parameter step is a pass of its own rather than the last product's epilogue:
// with 16 copies it moves 132 bytes an element, which the eight epilogue warps of
// a persistent product kernel cannot keep in flight (ResNet-50's last product took
// 972 us with the step in its epilogue, against 105 us without).  ResNet-50, 16 copies:
// momentum and norms 58 us (5.2 TB/s), planes 53 (5.8), parameter step 511 (6.6 of the
// measured 6.8).
#include "activation.cuh"
#include "ortho_kernels.h"
#include "product.h"
#include "tc_ptx.cuh"

namespace ddl {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = 4;  // groups of V elements whose loads a thread issues together

template <int V>
__device__ __forceinline__ void load_any(const void* base, int64_t at, int type, float (&v)[V]) {
  if (type == kF32) {
    const float* p = static_cast<const float*>(base) + at;
    if constexpr (V == 4) {
      const float4 u = *reinterpret_cast<const float4*>(p);
      v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    } else {
      v[0] = *p;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if constexpr (V == 4) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      const float2 a = from16x2(u.x, type), b = from16x2(u.y, type);
      v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    } else {
      v[0] = from16(*p, type);
    }
  }
}

template <int V>
__device__ __forceinline__ void store_any(void* base, int64_t at, int type, const float (&v)[V]) {
  if (type == kF32) {
    float* p = static_cast<float*>(base) + at;
    if constexpr (V == 4)
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *p = v[0];
  } else {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(p) = make_uint2(to16x2(v[0], v[1], type), to16x2(v[2], v[3], type));
    else
      *p = to16(v[0], type);
  }
}

// The groups of V elements of an item, in order of (row, column): group i's place.
struct Walk {
  uint32_t cols, total;  // groups in a row, in the item
  int32_t r0, c0;
  template <int V>
  static __device__ __forceinline__ Walk of(const OrthoItem& it) {
    const uint32_t cols = (uint32_t)(it.c1 - it.c0) / V;
    return {cols, cols * (uint32_t)(it.r1 - it.r0), it.r0, it.c0};
  }
  template <int V>
  __device__ __forceinline__ void place(const OrthoMatrix& m, uint32_t i, int64_t* flat, int64_t* plane) const {
    const uint32_t r = i / cols, c = (i - r * cols) * V + c0;
    *flat = m.offset + (int64_t)(r0 + r) * m.ld + c;
    *plane = (int64_t)(r0 + r) * m.ldp + c;
  }
};

// The sum over the CTA's threads, in a fixed order, for thread 0.  One warp does it: binary64 additions are slow here.
__device__ __forceinline__ double block_sum(double s) {
  __shared__ double part[kThreads];
  part[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = 0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) s += part[threadIdx.x + 32 * k];
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_down_sync(0xffffffffu, s, d);
  }
  return s;
}

// The sum of squares of an item whose squares may leave binary32's range, from what norms_item stored; out of line and
// rare.
__device__ __noinline__ double norms_in_64(const OrthoPrep* p, const OrthoMatrix* m, const OrthoItem* it) {
  const Walk walk = Walk::of<1>(*it);
  double s = 0;
  for (uint32_t i = threadIdx.x; i < walk.total; i += kThreads) {
    int64_t at, plane;
    walk.place<1>(*m, i, &at, &plane);
    float u[1], v[1];
    load_any(p->in, at, p->type, u);
    if (p->mom) {
      load_any(p->mom, at, kF32, v);
      u[0] = p->nesterov ? u[0] + p->mu * v[0] : v[0];
    }
    s += (double)u[0] * (double)u[0];
  }
  return s;
}

template <int V>
__device__ __forceinline__ double norms_item(const OrthoPrep& p, const OrthoMatrix& m, const OrthoItem& it) {
  const Walk walk = Walk::of<V>(it);
  // a thread's 32 or so squares in binary32, unless their size asks for binary64 (whose rate is low here)
  float sum = 0.f;
  bool wide = false;
  for (uint32_t i0 = threadIdx.x; i0 < walk.total; i0 += kThreads * kGroups) {
    int64_t at[kGroups];
    float g[kGroups][V], v[kGroups][V];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const uint32_t i = i0 + k * kThreads;
      if (i >= walk.total) continue;
      int64_t plane;
      walk.place<V>(m, i, &at[k], &plane);
      load_any(p.in, at[k], p.type, g[k]);
      if (p.mom) load_any(p.mom, at[k], kF32, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      if (i0 + k * kThreads >= walk.total) continue;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float u = g[k][j];
        if (p.mom) {
          v[k][j] = p.mu * v[k][j] + u;
          u = p.nesterov ? u + p.mu * v[k][j] : v[k][j];
        }
        const float a = fabsf(u);
        wide = wide || !(a < 1e18f) || (a < 1e-15f && a > 0.f);
        sum += u * u;
      }
      if (p.mom) store_any(p.mom, at[k], kF32, v[k]);
    }
  }
  // the barrier also puts the CTA's new momenta before the second reading
  return __syncthreads_or(wide) ? norms_in_64(&p, &m, &it) : (double)sum;
}

__global__ void __launch_bounds__(kThreads) norms_kernel(const __grid_constant__ OrthoPrep p) {
  const OrthoItem it = p.items[blockIdx.x];  // the handle's tables, written before any launch
  const OrthoMatrix m = p.matrices[it.matrix];
  tc::griddep_launch();
  tc::griddep_wait();
  const double s = block_sum(m.vec && p.vec ? norms_item<4>(p, m, it) : norms_item<1>(p, m, it));
  if (threadIdx.x == 0) p.partial[blockIdx.x] = s;
}

template <int V>
__device__ __forceinline__ void planes_item(const OrthoPrep& p, const OrthoMatrix& m, const OrthoItem& it, float power,
                                            float scale) {
  const Walk walk = Walk::of<V>(it);
  for (uint32_t i0 = threadIdx.x; i0 < walk.total; i0 += kThreads * kGroups) {
    int64_t plane[kGroups];
    float u[kGroups][V], v[kGroups][V];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const uint32_t i = i0 + k * kThreads;
      if (i >= walk.total) continue;
      int64_t at;
      walk.place<V>(m, i, &at, &plane[k]);
      if (!p.mom || p.nesterov) load_any(p.in, at, p.type, u[k]);
      if (p.mom) load_any(p.mom, at, kF32, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      if (i0 + k * kThreads >= walk.total) continue;
      float x[V], h[V], l[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float w = !p.mom ? u[k][j] : p.nesterov ? u[k][j] + p.mu * v[k][j] : v[k][j];
        x[j] = w * power * scale;
        h[j] = __half2float(__float2half_rn(x[j]));
        l[j] = x[j] - h[j];
      }
      store_any(m.hi[0], plane[k], kF16, h);
      store_any(m.lo[0], plane[k], kF16, l);
    }
  }
}

__global__ void __launch_bounds__(kThreads) planes_kernel(const __grid_constant__ OrthoPrep p) {
  __shared__ float power, inv;
  const OrthoItem it = p.items[blockIdx.x];  // the handle's tables, written before any launch
  const OrthoMatrix m = p.matrices[it.matrix];
  tc::griddep_launch();
  tc::griddep_wait();
  double s = 0;
  for (int i = threadIdx.x; i < m.n_items; i += kThreads) s += p.partial[m.item0 + i];
  s = block_sum(s);
  if (threadIdx.x == 0) {
    // of norms below 2^-60 (eps may be zero) a part of the factor is a power of two: binary32 would not hold the whole
    const double norm = sqrt(s) + (double)p.eps;
    power = norm < 0x1p-60 ? 0x1p60f : 1.f;
    inv = (float)((double)kPlaneScale / (norm * (double)power));
  }
  __syncthreads();
  if (m.vec && p.vec)
    planes_item<4>(p, m, it, power, inv);
  else
    planes_item<1>(p, m, it, power, inv);
}

template <int V>
__device__ __forceinline__ void finish_item(const OrthoFinish& p, const OrthoMatrix& m, const OrthoItem& it) {
  const Walk walk = Walk::of<V>(it);
  const float step = p.lr * m.shape_scale * (1.f / kPlaneScale);
  for (uint32_t i = threadIdx.x; i < walk.total; i += kThreads) {
    int64_t at, plane;
    walk.place<V>(m, i, &at, &plane);
    float x[V], l[V];
    load_any(m.hi[p.iterate], plane, kF16, x);
    load_any(m.lo[p.iterate], plane, kF16, l);
    if (!p.out) {
#pragma unroll 1
      for (int c = 0; c < p.n_copies; c += 4) {
        float t[4][V];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (c + k < p.n_copies) load_any(p.copies[c + k], at, kF32, t[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (c + k >= p.n_copies) break;
#pragma unroll
          for (int j = 0; j < V; ++j) t[k][j] = t[k][j] * p.decay - step * (x[j] + l[j]);
          store_any(p.copies[c + k], at, kF32, t[k]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = (x[j] + l[j]) * (1.f / kPlaneScale);
      store_any(p.out, at, p.type, x);
    }
  }
}

__global__ void __launch_bounds__(kThreads) finish_kernel(const __grid_constant__ OrthoFinish p) {
  const OrthoItem it = p.items[blockIdx.x];  // the handle's tables, written before any launch
  const OrthoMatrix m = p.matrices[it.matrix];
  tc::griddep_launch();
  tc::griddep_wait();
  if (m.vec && p.vec)
    finish_item<4>(p, m, it);
  else
    finish_item<1>(p, m, it);
}

}  // namespace

cudaError_t launch_ortho_norms(const OrthoPrep& p, cudaStream_t stream) {
  return tc::launch_early(norms_kernel, dim3((unsigned)p.n_items), kThreads, stream, p);
}

cudaError_t launch_ortho_planes(const OrthoPrep& p, cudaStream_t stream) {
  return tc::launch_early(planes_kernel, dim3((unsigned)p.n_items), kThreads, stream, p);
}

cudaError_t launch_ortho_finish(const OrthoFinish& p, cudaStream_t stream) {
  return tc::launch_early(finish_kernel, dim3((unsigned)p.n_items), kThreads, stream, p);
}

}  // namespace ddl
