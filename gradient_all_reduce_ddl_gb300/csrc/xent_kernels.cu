// xent_kernels.cu -- the passes around the products of the softmax cross entropy:
// joining the vocabulary's parts, the planes' scale of many tokens, and, in one
// launch, the bias gradient and the rounding of dx's sums.  All of them read what the products left in L2, and
// small calls are bound by their launches (a join 3 us in a sequence).  8192 tokens x 512
// parts are joined in 14 us, 8192 x 2048 sums rounded with the label's correction in 22 (cold; 4.5 TB/s).
#include <cfloat>

#include "activation.cuh"
#include "product.h"
#include "tc_ptx.cuh"
#include "xent.cuh"
#include "xent_kernels.h"

namespace ddl {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// sum exp(z - most) over parts of it
struct LogSum {
  float most, sum;
  __device__ __forceinline__ void add(float m, float s) {
    const float top = fmaxf(most, m);
    // equal ones, infinite ones among them, keep their sums; a NaN in a sum stays
    sum = sum * (most == top ? 1.f : expf(most - top)) + s * (m == top ? 1.f : expf(m - top));
    most = top;
  }
};

// TX tokens per CTA (1, 8 or 32), its other threads share out the parts: those of a warp join by shuffles, the warps through
// shared memory.
template <int TX>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ XentJoin p) {
  constexpr int TY = kThreads / TX, kBatch = TX == 32 ? 8 : 4;
  __shared__ float2 shared[kWarps][TX];
  __shared__ float shared_sum[kWarps][TX];
  tc::griddep_launch();
  tc::griddep_wait();
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * TX + tx;
  const bool in = t < p.tokens, writes = ty == 0 && in;
  int64_t y = -1;
  float z = 0.f;
  if (writes) {
    y = p.labels[t];
    z = __ldcg(p.picked + t);  // not set without a label
  }
  LogSum l = {-INFINITY, 0.f};
  float all = 0.f;
  if (in) {
    for (int k0 = ty; k0 < p.n_parts; k0 += kBatch * TY) {
      float2 u[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        u[k] = k0 + k * TY < p.n_parts ? __ldcg(p.part + (int64_t)(k0 + k * TY) * p.ld + t) : make_float2(-INFINITY, 0.f);
      // as add(), of all of them
      float most = l.most, s = 0.f;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) most = fmaxf(most, u[k].x);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) s += u[k].y * (u[k].x == most ? 1.f : expf(u[k].x - most));
      l.sum = l.sum * (l.most == most ? 1.f : expf(l.most - most)) + s;
      l.most = most;
    }
    if (p.part_sum) {
#pragma unroll 4
      for (int k = ty; k < p.n_parts; k += TY) all += __ldcg(p.part_sum + (int64_t)k * p.ld + t);
    }
  }
#pragma unroll
  for (int d = 16; d >= TX; d >>= 1) {
    const float m = __shfl_xor_sync(0xFFFFFFFFu, l.most, d), s = __shfl_xor_sync(0xFFFFFFFFu, l.sum, d);
    l.add(m, s);
    all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
  }
  if ((threadIdx.x & 31) < TX) {
    shared[warp][tx] = make_float2(l.most, l.sum);
    shared_sum[warp][tx] = all;
  }
  __syncthreads();
  if (!writes) return;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) {
    const float2 u = shared[w][tx];
    l.add(u.x, u.y);
    all += shared_sum[w][tx];
  }
  float loss = 0.f, lse;
  if (y < 0 || y >= p.vocab) {
    lse = l.most + logf(l.sum);
    if (y >= p.vocab) {
      loss = NAN;
      atomicOr(p.err, kErrLabel);
    }
  } else {
    // lse - z, with z the label's logit: what the others add to it, or what is left of them
    loss = z >= l.most ? log1pf(l.sum * expf(l.most - z)) : (l.most - z) + logf(l.sum + expf(z - l.most));
    LogSum every = l;
    every.add(z, 1.f);
    lse = every.most + logf(every.sum);
    if (p.part_sum) loss += p.smoothing * (z - all / ((float)p.vocab * kSumScale));
  }
  if (p.loss) p.loss[t] = loss;
  if (p.lse) p.lse[t] = lse;
}

__global__ void __launch_bounds__(1024) scale_kernel(const __grid_constant__ XentScale p) {
  __shared__ uint32_t shared[2][32];
  tc::griddep_launch();
  tc::griddep_wait();
  uint32_t most = 0, counted = 0;
  for (int64_t t = threadIdx.x; t < p.tokens; t += 1024) {
    const uint32_t b = coef_bits(p.coef, p.labels, t, p.vocab);
    most = max(most, b);
    counted += b != 0;
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  counted = __reduce_add_sync(0xFFFFFFFFu, counted);
  if ((threadIdx.x & 31) == 0) shared[0][threadIdx.x >> 5] = most, shared[1][threadIdx.x >> 5] = counted;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  most = __reduce_max_sync(0xFFFFFFFFu, shared[0][threadIdx.x]);
  counted = __reduce_add_sync(0xFFFFFFFFu, shared[1][threadIdx.x]);
  if (threadIdx.x == 0) {
    const float2 u = dz_scale(most, p.f16);
    p.scale[0] = u.x, p.scale[1] = u.y, p.scale[2] = __int_as_float(planes_of(counted, p.planes));
  }
}

__device__ __forceinline__ void bias_columns(const XentBias& p, int64_t block) {
  __shared__ float shared[kWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = block * 32 + lane;
  float s = 0.f;
  if (c < p.cols) {
#pragma unroll 4
    for (int64_t g = warp; g < p.groups; g += kWarps) s += __ldcg(p.part + g * p.ld + c);
  }
  shared[warp][lane] = s;
  __syncthreads();
  if (warp > 0 || c >= p.cols) return;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) s += shared[w][lane];
  s *= __ldcg(p.scale);
  if (p.f32) {
    float* o = static_cast<float*>(p.db) + c;
    *o = p.accumulate ? *o + s : s;
  } else {
    __half* o = static_cast<__half*>(p.db) + c;
    *o = __float2half_rn(p.accumulate ? __half2float(*o) + s : s);
  }
}

__device__ __forceinline__ void round_rows(const XentRound& p, int64_t block) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t across = (p.cols + 255) / 256;
  const int64_t r = block / across * kWarps + warp, c0 = block % across * 256 + lane;
  if (r >= p.rows) return;
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = c0 + 32 * k < p.cols ? __ldcs(p.src + r * p.ld + c0 + 32 * k) : 0.f;
  const int64_t y = p.labels[r];
  if (y >= 0 && y < p.vocab) {
    const float by = __ldcg(p.resid + r) * __ldcg(p.inverse);
    uint16_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = c0 + 32 * k < p.cols ? p.w[y * p.ldw + c0 + 32 * k] : 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // (an infinite or NaN sum stands: the rest, or its zero, times the weight that made it so may be NaN)
      const float u = fmaf(by, from16(w[k], p.type), v[k]);
      v[k] = fabsf(v[k]) <= FLT_MAX ? u : v[k];
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (c0 + 32 * k < p.cols) p.dst[r * p.ldd + c0 + 32 * k] = to16(v[k], p.type);
}

int64_t bias_blocks(const XentBias& p) { return p.db ? (p.cols + 31) / 32 : 0; }

__global__ void __launch_bounds__(kThreads) end_kernel(const __grid_constant__ XentEnd p, uint32_t first) {
  tc::griddep_launch();
  tc::griddep_wait();
  if (blockIdx.x < first)
    bias_columns(p.bias, blockIdx.x);
  else
    round_rows(p.round, blockIdx.x - first);
}

}  // namespace

cudaError_t launch_xent_join(const XentJoin& p, cudaStream_t stream) {
  if (p.tokens >= 1024) return tc::launch_early(join_kernel<32>, dim3((unsigned)((p.tokens + 31) / 32)), kThreads, stream, p);
  if (p.tokens >= 64) return tc::launch_early(join_kernel<8>, dim3((unsigned)((p.tokens + 7) / 8)), kThreads, stream, p);
  return tc::launch_early(join_kernel<1>, dim3((unsigned)p.tokens), kThreads, stream, p);
}

cudaError_t launch_xent_scale(const XentScale& p, cudaStream_t stream) {
  return tc::launch_early(scale_kernel, dim3(1), 1024, stream, p);
}

cudaError_t launch_xent_end(const XentEnd& p, cudaStream_t stream) {
  const int64_t first = bias_blocks(p.bias), blocks = first + (p.round.rows + kWarps - 1) / kWarps * ((p.round.cols + 255) / 256);
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return tc::launch_early(end_kernel, dim3((unsigned)blocks), kThreads, stream, p, (uint32_t)first);
}

}  // namespace ddl
