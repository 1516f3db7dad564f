// adam_kernels.cu -- the AdamW step over many tensors of a flat buffer, on every
// worker's copy of the parameters, and the gradient's norm.
//
//   g' = c g;   m = b1 m + (1 - b1) g';   v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Bound by HBM: 28 bytes an element with binary32 states and one copy, 8 (10 with a
// 16-bit operand copy) for each further copy; 16.1 with 8-bit states, whose coding also
// takes 69 instructions an element (56 % of the issue slots).  One launch covers every tensor: a CTA takes an
// item of up to 1024 elements of one tensor, each of its warps one or two
// neighbouring blocks of 128, four elements per lane, so that a block's largest value (the
// 8-bit states' scale) is one warp reduction, the work does not depend on how long the
// tensors are, and what the SMs have in flight lies together (warps that walk 1024 elements
// each on their own: 1720 us for the 336 M elements below).
//
// Products and sums are rounded one by one (no fused multiply-adds), as in the fused
// SGD update, so that binary32 states are the same bits as in a step-by-step evaluation; of
// 8-bit ones a code can be the neighbour's where the root lies next to the middle of two.
#include <cuda_fp8.h>

#include "activation.cuh"
#include "adam_kernels.h"
#include "tc_ptx.cuh"

namespace ddl {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr float kTop = 448.f;             // e4m3's largest number
constexpr float kLeast = 0x1p-100f;       // blocks whose largest value is below this are kept as zeros
constexpr uint32_t kCodeNan = 0x7F;

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
__device__ __forceinline__ uint32_t load_codes(const void* base, int64_t at, uint32_t len, int lane) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + at;
  if constexpr (V == 4) return *reinterpret_cast<const uint32_t*>(p + 4 * lane);
  uint32_t u = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (place<V>(lane, j) < len) u |= (uint32_t)p[place<V>(lane, j)] << (8 * j);
  return u;
}

__device__ __forceinline__ void decode(uint32_t u, float scale, float (&x)[4]) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u & 0xFFFFu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> 16), __NV_E4M3);
  const float2 f = __half22float2(__half2(a)), g = __half22float2(__half2(b));
  x[0] = f.x * scale, x[1] = f.y * scale, x[2] = g.x * scale, x[3] = g.y * scale;
}

// Encodes a block's values (zeros outside the tensor; ROOT: none negative) and returns its scale.
template <int V, bool ROOT>
__device__ __forceinline__ float store_codes(void* base, int64_t at, uint32_t len, int lane, const float (&x)[4]) {
  // the largest magnitude: as bits they order as the numbers do
  constexpr uint32_t kSign = ROOT ? 0xFFFFFFFFu : 0x7FFFFFFFu, kInf = 0x7F800000u;
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(x[j]) & kSign;
  uint32_t most = __reduce_max_sync(0xFFFFFFFFu, max(max(b[0], b[1]), max(b[2], b[3])));
  const bool finite = most < kInf;
  if (!finite) {  // the largest of the others
    most = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((b[j] & 0x7FFFFFFFu) < kInf) most = max(most, b[j]);
    most = __reduce_max_sync(0xFFFFFFFFu, most);
  }
  const float top = __uint_as_float(most);
  const bool held = top >= kLeast;
  const float by = held ? kTop / top : 0.f;
  float y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    y[j] = x[j] * by;
    if (ROOT && held && x[j] > 0.f) y[j] = fmaxf(y[j], 0x1p-9f);
  }
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
  uint32_t u = (uint32_t)lo | (uint32_t)hi << 16;
  if (!finite) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((b[j] & 0x7FFFFFFFu) >= kInf) u = (u & ~(0xFFu << (8 * j))) | kCodeNan << (8 * j);
  }
  uint8_t* p = static_cast<uint8_t*>(base) + at;
  if constexpr (V == 4) {
    *reinterpret_cast<uint32_t*>(p + 4 * lane) = u;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (place<V>(lane, j) < len) p[place<V>(lane, j)] = (uint8_t)(u >> (8 * j));
  }
  return held ? top * (1.f / kTop) : 0.f;
}

// -- the step -----------------------------------------------------------------------

// Occupancy and grid, by the states' width.  336 M elements with 8-bit states, the norm's pass among them: seven CTAs of 128
// threads an SM (72 registers) 1222 us (1190 since roots are scaled, see below), eight (64, some spilled) 1248, six 1231, four of
// 256 threads 1272, three 1286; loads of the next item before this one's arithmetic 1277 (112 registers), one block at a time
// instead of two 1460.  25.6 M elements of 16 copies with binary32 states: a grid of four times the CTAs that fit 565 us, of those
// that fit 576.
__host__ __device__ constexpr int min_ctas(int bits) { return bits == 32 ? 6 : 7; }
constexpr int waves(int bits) { return bits == 32 ? 24 : 7; }

// What the step count and the norm make of the parameters, in every thread.
struct Factors {
  float scale;  // of the gradient
  float size;   // lr / (1 - b1^t)
  float root;   // 1 / sqrt(1 - b2^t)
};

// To 2 units in the last place, also of numbers below the normal range, which the instruction takes for 0.  The roots are stored in
// 8 bits or not at all, and the step is far below the parameter.  (Correctly rounded: 336 M elements 1188 -> 1271 us.)
__device__ __forceinline__ float root_of(float x) {
  const bool low = x < 0x1p-100f;
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(low ? x * 0x1p64f : x));
  return low ? y * 0x1p-32f : y;
}
__device__ __forceinline__ float inverse_of(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// This warp's part [first, end) of an item: a block of each four, or two neighbours of each eight.
__device__ __forceinline__ void share_of(const AdamItem& it, uint32_t* first, uint32_t* end) {
  const uint32_t share = it.len > kWarps * kAdamBlock ? 2 * kAdamBlock : kAdamBlock;
  *first = (threadIdx.x >> 5) * share;
  *end = *first + share < it.len ? *first + share : it.len;
}

// NB blocks of 128 elements in a row (V = 1: one, of len elements), whose loads are all issued before the first is used.
template <int BITS, int V, int NB, class Copies>
__device__ __forceinline__ void blocks_step(const AdamStep& p, const Copies& to, const Factors& f, const AdamItem& it, uint32_t first,
                                            uint32_t len, int lane) {
  const int64_t at0 = (int64_t)(it.begin + first);
  const uint32_t block = it.block + first / kAdamBlock;
  constexpr int kCopies = BITS == 32 ? 2 : 1;  // in flight
  float g[NB][4], m[NB][4], v[NB][4], t[kCopies][NB][4], sm[NB], sv[NB];
  uint32_t cm[NB], cv[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t at = at0 + b * kAdamBlock;
    load_grad<V>(p.grad, at, p.grad_type, len, lane, g[b]);
    if constexpr (BITS == 32) {
      load32<V>(static_cast<const float*>(p.m) + at, len, lane, m[b]);
      load32<V>(static_cast<const float*>(p.v) + at, len, lane, v[b]);
    } else {
      cm[b] = load_codes<V>(p.m, at, len, lane), cv[b] = load_codes<V>(p.v, at, len, lane);
      sm[b] = p.scale_m[block + b], sv[b] = p.scale_v[block + b];
    }
  }
#pragma unroll
  for (int k = 0; k < kCopies; ++k)
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (k < p.n_copies) load32<V>(to.params[k] + at0 + b * kAdamBlock, len, lane, t[k][b]);
  const float size = f.size * it.lr, keep = 1.f - p.lr * it.lr * p.weight_decay * it.decay;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int64_t at = at0 + b * kAdamBlock;
    if constexpr (BITS == 8) {
      decode(cm[b], sm[b], m[b]);
      decode(cv[b], sv[b], v[b]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[b][j] *= v[b][j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = g[b][j] * f.scale;
      m[b][j] = m[b][j] * p.beta1 + x * p.rest1;
      v[b][j] = v[b][j] * p.beta2 + x * p.rest2 * x;
      const float root = root_of(v[b][j]);
      g[b][j] = m[b][j] * size * inverse_of(root * f.root + p.eps);
      if (BITS == 8) v[b][j] = root;
    }
    if constexpr (BITS == 32) {
      store32<V>(static_cast<float*>(p.m) + at, len, lane, m[b]);
      store32<V>(static_cast<float*>(p.v) + at, len, lane, v[b]);
    } else {
      sm[b] = store_codes<V, false>(p.m, at, len, lane, m[b]);
      sv[b] = store_codes<V, true>(p.v, at, len, lane, v[b]);
      if (lane == 0) p.scale_m[block + b] = sm[b], p.scale_v[block + b] = sv[b];
    }
  }
#pragma unroll 1
  for (int c = 0; c < p.n_copies; c += kCopies) {
    if (c > 0) {
#pragma unroll
      for (int k = 0; k < kCopies; ++k)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          if (c + k < p.n_copies) load32<V>(to.params[c + k] + at0 + b * kAdamBlock, len, lane, t[k][b]);
    }
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      if (c + k >= p.n_copies) break;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int64_t at = at0 + b * kAdamBlock;
#pragma unroll
        for (int j = 0; j < 4; ++j) t[k][b][j] = t[k][b][j] * keep - g[b][j];
        store32<V>(to.params[c + k] + at, len, lane, t[k][b]);
        if (p.operands) store16<V>(to.out[c + k], at, p.out_type, len, lane, t[k][b]);
      }
    }
  }
}

// ODD: some buffer or tensor does not begin at a multiple of four elements.  Its path takes registers that the other kernel
// would spill (336 M elements 1440 instead of 1198 us), and two blocks at a time, too (2.3 M elements of odd tensors 14.2 ->
// 11.8 us).
template <int BITS, int COPIES, bool ODD>
__global__ void __launch_bounds__(kThreads, min_ctas(BITS))
    step_kernel(const __grid_constant__ AdamStep p, const __grid_constant__ AdamCopies<COPIES> to) {
  const int lane = threadIdx.x & 31;
  AdamItem next = p.items[blockIdx.x];  // the handle's table, written before any launch
  tc::griddep_launch();
  tc::griddep_wait();
  const int64_t t = *p.step + 1;
  Factors f;
  // 1 - b^t = -expm1(t log b): the difference would lose what is left of a beta near one
  f.size = p.lr / -expm1f((float)((double)t * p.log_beta1));
  f.root = 1.f / sqrtf(-expm1f((float)((double)t * p.log_beta2)));
  f.scale = p.norm ? p.norm->scale : p.grad_scale;
  for (int64_t i = blockIdx.x; i < p.n_items; i += gridDim.x) {
    const AdamItem it = next;
    if (i + gridDim.x < p.n_items) next = p.items[i + gridDim.x];
    uint32_t first, end;
    share_of(it, &first, &end);
    if (p.vec && it.begin % 4 == 0) {
      if (first + 2 * kAdamBlock <= end) {
        blocks_step<BITS, 4, 2>(p, to, f, it, first, kAdamBlock, lane);
        continue;
      }
      if (first + kAdamBlock <= end) {
        blocks_step<BITS, 4, 1>(p, to, f, it, first, kAdamBlock, lane);
        first += kAdamBlock;
      }
    } else if (ODD && first + 2 * kAdamBlock <= end) {
      blocks_step<BITS, 1, 2>(p, to, f, it, first, kAdamBlock, lane);
      continue;
    }
#pragma unroll 1
    for (; first < end; first += kAdamBlock)
      blocks_step<BITS, 1, 1>(p, to, f, it, first, end - first < kAdamBlock ? end - first : kAdamBlock, lane);
  }
  // the last CTA counts the step: every other one has read the count
  __syncthreads();
  if (threadIdx.x == 0 && atomicInc(p.done, gridDim.x - 1) == gridDim.x - 1) *p.step = t;
}

// -- the gradient's norm ---------------------------------------------------------------

// A sum of squares: in two binary32 numbers, what the first one's additions lose kept in the second (binary64 additions
// would bound the pass: 404 against 194 us of 336 M elements, 6.9 TB/s), and squares outside of binary32's range in binary64.
struct Squares {
  float sum = 0.f, lost = 0.f;
  double far = 0.0;
  __device__ __forceinline__ void add(const float (&g)[4]) {
    const float x = (g[0] * g[0] + g[1] * g[1]) + (g[2] * g[2] + g[3] * g[3]);
    if (x > 0x1p-80f && x < 0x1p100f) {
      const float t = sum + x, part = t - sum;
      lost += (sum - (t - part)) + (x - part);
      sum = t;
    } else if (g[0] != 0.f || g[1] != 0.f || g[2] != 0.f || g[3] != 0.f) {
#pragma unroll
      for (int j = 0; j < 4; ++j) far += (double)g[j] * (double)g[j];
    }
  }
  __device__ __forceinline__ double value() const { return (double)sum + (double)lost + far; }
};

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
  AdamItem next = p.items[blockIdx.x];  // the handle's table, written before any launch
  tc::griddep_launch();
  tc::griddep_wait();
  Squares q;
  for (int64_t i = blockIdx.x; i < p.n_items; i += gridDim.x) {
    const AdamItem it = next;
    if (i + gridDim.x < p.n_items) next = p.items[i + gridDim.x];
    uint32_t first, end;
    share_of(it, &first, &end);
    float g[2][4] = {};
    if (p.vec && it.begin % 4 == 0 && first + 2 * kAdamBlock <= end) {
      load_grad<4>(p.grad, (int64_t)(it.begin + first), p.grad_type, kAdamBlock, lane, g[0]);
      load_grad<4>(p.grad, (int64_t)(it.begin + first) + kAdamBlock, p.grad_type, kAdamBlock, lane, g[1]);
    } else if (first < end) {
      load_grad<1>(p.grad, (int64_t)(it.begin + first), p.grad_type, end - first, lane, g[0]);
      if (first + kAdamBlock < end)
        load_grad<1>(p.grad, (int64_t)(it.begin + first) + kAdamBlock, p.grad_type, end - first - kAdamBlock, lane, g[1]);
    }
    q.add(g[0]);
    q.add(g[1]);
  }
  double s = q.value();
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
  const int64_t wave = (int64_t)sms * most;
  return (unsigned)(p.n_items < wave ? p.n_items : wave);
}

template <int COPIES>
cudaError_t launch_copies(const AdamStep& p, const AdamCopies<COPIES>& c, int sms, cudaStream_t stream) {
  const dim3 grid(grid_of(p, sms, waves(p.bits)));
  if (p.bits == 8)
    return p.odd ? tc::launch_early(step_kernel<8, COPIES, true>, grid, kThreads, stream, p, c)
                 : tc::launch_early(step_kernel<8, COPIES, false>, grid, kThreads, stream, p, c);
  return p.odd ? tc::launch_early(step_kernel<32, COPIES, true>, grid, kThreads, stream, p, c)
               : tc::launch_early(step_kernel<32, COPIES, false>, grid, kThreads, stream, p, c);
}

}  // namespace

cudaError_t launch_adam_norm(const AdamStep& p, int sms, cudaStream_t stream) {
  unsigned grid = grid_of(p, sms, 12);
  if (grid > kMaxNormParts) grid = kMaxNormParts;
  return tc::launch_early(norm_kernel, dim3(grid), kThreads, stream, p);
}

cudaError_t launch_adam_step(const AdamStep& p, const AdamCopies<kMaxAdamCopies>& c, int sms, cudaStream_t stream) {
  if (p.n_copies > kFewAdamCopies) return launch_copies(p, c, sms, stream);
  AdamCopies<kFewAdamCopies> few = {};
  for (int k = 0; k < p.n_copies; ++k) few.params[k] = c.params[k], few.out[k] = c.out[k];
  return launch_copies(p, few, sms, stream);
}

}  // namespace ddl
