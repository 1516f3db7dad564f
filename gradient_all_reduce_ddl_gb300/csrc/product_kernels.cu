// product_kernels.cu -- the tensor-core product kernel of the linear layers
// and of the Newton-Schulz steps.
//
//   D(i, j) = sum_pass scale_pass sum_k A_pass(i, k) B_pass(j, k)
//
// on tcgen05 (128 x tile_n tiles, accumulators in TMEM), then one of the
// epilogues of product.h.
//
// Roles of a CTA's ten warps: warp 0 loads operand boxes by TMA into a ring
// of shared-memory stages, warp 1 issues the products, warps 2-9 take the
// finished sums out of TMEM, add them in binary32 registers, pass them through
// shared memory (so that every global access of the epilogue runs along rows)
// and write the result.  The two TMEM accumulators alternate, so the epilogue
// of one chunk or tile runs under the products of the next.
//
// The tensor core adds with truncation: a long sum of one sign loses about
// half a unit in the last place of each of its K/16 additions.  Results kept in
// binary32 therefore leave the accumulator every `chunk` K blocks and are added
// in registers with rounding to nearest; 16-bit results sum all of K in TMEM.
//
// A long contraction with few tiles is split over the CTAs of a cluster; each
// leaves its sums in shared memory and the cluster's CTAs add them in rank order
// through distributed shared memory, so results do not depend on timing.
//
// Every wait is bounded.  One that runs out sets kErrProductWait; the CTA then
// waits (bounded too) for its own loads and products, frees its TMEM and ends.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "product.h"
#include "tc_ptx.cuh"

namespace ddl {
namespace {

using namespace tc;

constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kBoxBytes = kBoxRows * kBlockK * 2;
constexpr int kABytes = kTileM * kBlockK * 2;
constexpr float kLoScale = 2048.f;  // lo planes hold (x - hi) * 2^11

__host__ __device__ constexpr int stages(int bn) { return bn == 128 ? 4 : 6; }
__host__ __device__ constexpr int stage_bytes(int bn) { return kABytes + bn * kBlockK * 2; }
__host__ __device__ constexpr int pitch(int bn) { return bn + 4; }  // floats; rows 4 banks apart
__host__ __device__ constexpr int smem_bytes(int bn) {
  return 1024 + stages(bn) * stage_bytes(bn) + kTileM * pitch(bn) * 4;
}

// -- element access -------------------------------------------------------------

__device__ __forceinline__ float from16(uint16_t u, int type) {
  return type == kBF16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
}
__device__ __forceinline__ uint16_t to16(float x, int type) {
  return type == kBF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

template <int V>
__device__ __forceinline__ void load16(const void* base, int64_t at, int type, float (&v)[V]) {
  const uint16_t* p = static_cast<const uint16_t*>(base) + at;
  if constexpr (V == 4) {
    const ushort4 u = *reinterpret_cast<const ushort4*>(p);
    v[0] = from16(u.x, type), v[1] = from16(u.y, type), v[2] = from16(u.z, type), v[3] = from16(u.w, type);
  } else {
    v[0] = from16(*p, type);
  }
}

template <int V>
__device__ __forceinline__ void store16(void* base, int64_t at, int type, const float (&v)[V]) {
  uint16_t* p = static_cast<uint16_t*>(base) + at;
  if constexpr (V == 4)
    *reinterpret_cast<ushort4*>(p) = make_ushort4(to16(v[0], type), to16(v[1], type), to16(v[2], type), to16(v[3], type));
  else
    *p = to16(v[0], type);
}

template <int V>
__device__ __forceinline__ void load32(const float* p, float (&v)[V]) {
  if constexpr (V == 4) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  } else {
    v[0] = *p;
  }
}

template <int V>
__device__ __forceinline__ void store32(float* p, const float (&v)[V]) {
  if constexpr (V == 4)
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *p = v[0];
}

template <int V>
__device__ __forceinline__ void load_any(const void* base, int64_t at, int type, float (&v)[V]) {
  if (type == kF32)
    load32(static_cast<const float*>(base) + at, v);
  else
    load16(base, at, type, v);
}

template <int V>
__device__ __forceinline__ void store_any(void* base, int64_t at, int type, const float (&v)[V]) {
  if (type == kF32)
    store32(static_cast<float*>(base) + at, v);
  else
    store16(base, at, type, v);
}

// x ~ hi + 2^-11 lo, 22 bits of x while hi is a normal binary16 (below that the
// error stays under 2^-36); an infinite or NaN hi carries the value alone.
__device__ __forceinline__ void split(float x, uint16_t* hi, uint16_t* lo) {
  const __half h = __float2half_rn(x);
  const float hf = __half2float(h);
  *hi = __half_as_ushort(h);
  *lo = isfinite(hf) ? __half_as_ushort(__float2half_rn((x - hf) * kLoScale)) : (uint16_t)0;
}

template <int V>
__device__ __forceinline__ void store_planes(uint16_t* hi, uint16_t* lo, int64_t at, const float (&v)[V]) {
  uint16_t h[V], l[V];
#pragma unroll
  for (int k = 0; k < V; ++k) split(v[k], &h[k], &l[k]);
  if constexpr (V == 4) {
    *reinterpret_cast<ushort4*>(hi + at) = make_ushort4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<ushort4*>(lo + at) = make_ushort4(l[0], l[1], l[2], l[3]);
  } else {
    hi[at] = h[0];
    lo[at] = l[0];
  }
}

template <int V>
__device__ __forceinline__ void load_planes(const uint16_t* hi, const uint16_t* lo, int64_t at, float (&v)[V]) {
  float l[V];
  load16(hi, at, kF16, v);
  load16(lo, at, kF16, l);
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] += l[k] * (1.f / kLoScale);
}

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.f ? z : (z != z ? z : 0.f);
    case kActGelu: return z * (0.5f * (1.f + erff(z * 0.70710678118654752f)));
    case kActSilu: return z / (1.f + expf(-z));
    default: return z;
  }
}

// -- epilogues: V values of D that belong at output row m, columns n.. ------------

template <int V, bool GROUPED>
__device__ __forceinline__ void emit(const Product& P, const ProductLaunch& p, int m, int n, float (&v)[V]) {
  if constexpr (!GROUPED) {
    if (P.epi == kEpiLinear) {
      float t[V];
      if (P.bias) {
        load16(P.bias, n, P.type, t);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] += t[k];
      }
      if (P.z) store16(P.z, (int64_t)m * P.ldz + n, P.type, v);
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = activate(v[k], P.act);
      if (P.add) {
        load16(P.add, (int64_t)m * P.ld_add + n, P.type, t);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] += t[k];
      }
      store16(P.out, (int64_t)m * P.ldo + n, P.type, v);
    } else {
      const int64_t at = (int64_t)m * P.ldo + n;
      if (P.accumulate) {
        float t[V];
        load_any(P.out, at, P.out_type, t);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] += t[k];
      }
      store_any(P.out, at, P.out_type, v);
    }
  } else {
    if (P.epi == kEpiGram) {
      store_planes(P.p_hi, P.p_lo, (int64_t)m * P.ldp + n, v);
      return;
    }
    float c[V];
    load_planes(P.c_hi, P.c_lo, (int64_t)m * P.ldc + n, c);
    if (P.epi == kEpiPoly) {
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = p.cb * c[k] + p.cc * v[k];
      store_planes(P.p_hi, P.p_lo, (int64_t)m * P.ldp + n, v);
      return;
    }
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = p.ca * c[k] + v[k];
    if (P.epi == kEpiApply) {
      store_planes(P.p_hi, P.p_lo, (int64_t)m * P.ldp + n, v);
      return;
    }
    const int64_t at = P.offset + (int64_t)m * P.ldo + n;
    if (p.last_epi == kEpiOrtho) {
      store_any(p.flat_out, at, p.flat_type, v);
      return;
    }
    const float step = p.lr * P.shape_scale;
    for (int r = 0; r < p.n_copies; r += 4) {  // four copies' loads in flight
      float t[4][V];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (r + j < p.n_copies) load32(p.copies[r + j] + at, t[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (r + j < p.n_copies) {
#pragma unroll
          for (int k = 0; k < V; ++k) t[j][k] = t[j][k] * p.decay - step * v[k];
          store32(p.copies[r + j] + at, t[j]);
        }
    }
  }
}

struct Place {
  const Product* P;
  int row0, col0, mirror;
};

// Whether a product's epilogue may take 4 elements at a time.
template <bool GROUPED>
__device__ __forceinline__ bool wide_access(const Product& P, const ProductLaunch& p) {
  return P.vec && (!GROUPED || P.epi != kEpiOrtho || p.flat_vec);
}

template <int BN, bool GROUPED>
__device__ __forceinline__ Place place(const ProductLaunch& p, int t) {
  if constexpr (GROUPED) {
    const int4 u = __ldg(reinterpret_cast<const int4*>(p.g_tiles) + t);
    return {p.g_products + u.x, u.y * kTileM, u.z * BN, u.w};
  } else {
    int k = 0;
    if (t >= p.inl_tiles[0]) {
      k = 1;
      t -= p.inl_tiles[0];
    }
    const Product* P = &p.inl[k];
    // bands of 16 tile rows, column by column, so that CTAs in flight share operands in L2
    const int rows = (P->M + kTileM - 1) / kTileM, cols = (P->N + BN - 1) / BN;
    const int band = t / (16 * cols), first = band * 16;
    const int height = rows - first < 16 ? rows - first : 16;
    const int in = t - band * 16 * cols;
    return {P, (first + in % height) * kTileM, in / height * BN, 0};
  }
}

template <int BN, bool GROUPED>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ ProductLaunch p) {
  constexpr int kStages = stages(BN);
  constexpr int kPitch = pitch(BN);
  constexpr uint32_t kCols = 2 * BN;
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bars[2 * kStages + 5];
  __shared__ uint32_t tmem_slot;
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t staging = ring + kStages * stage_bytes(BN);
  const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages, tempty = tfull + 16,
                 drain = tempty + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(full + 8 * s, 1);
      bar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(tfull + 8 * b, 1);
      bar_init(tempty + 8 * b, kEpiWarps);
    }
    bar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), kCols);
    fence_before();
  }
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;
  griddep_launch();
  griddep_wait();

  const int S = p.splits;
  const int q = S > 1 ? (int)cluster_rank() : 0;
  const int first = blockIdx.x / S, step = gridDim.x / S;
  const CUtensorMap* maps = GROUPED ? p.g_maps : p.maps;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = first; t < p.n_tiles && ok; t += step) {
        const Place pl = place<BN, GROUPED>(p, t);
        const Product& P = *pl.P;
        const int nkb = (P.K + kBlockK - 1) / kBlockK, kb0 = nkb * q / S, kb1 = nkb * (q + 1) / S;
        for (int ps = 0; ps < P.n_pass && ok; ++ps) {
          const CUtensorMap* ma = maps + P.a[ps];
          const CUtensorMap* mb = maps + P.b[ps];
          if constexpr (GROUPED) {  // written by the host before this launch
            asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(ma) : "memory");
            asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(mb) : "memory");
          }
          for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const uint32_t s = it % kStages;
            if (!bar_wait(empty + 8 * s, (it / kStages & 1u) ^ 1u)) {
              atomicOr(p.err, kErrProductWait);
              ok = false;
              break;
            }
            const uint32_t sa = ring + s * stage_bytes(BN), sb = sa + kABytes, bar = full + 8 * s;
            bar_expect(bar, stage_bytes(BN));
#pragma unroll
            for (int h = 0; h < kTileM / kBoxRows; ++h) {
              const int row = pl.row0 + h * kBoxRows;
              tma_box(sa + h * kBoxBytes, ma, bar, P.a_mn ? row : kb * kBlockK, P.a_mn ? kb * kBlockK : row);
            }
#pragma unroll
            for (int h = 0; h < (BN + kBoxRows - 1) / kBoxRows; ++h) {
              const int row = pl.col0 + h * kBoxRows;
              tma_box(sb + h * kBoxBytes, mb, bar, P.b_mn ? row : kb * kBlockK, P.b_mn ? kb * kBlockK : row);
            }
          }
        }
      }
      // loads in flight end before the CTA does
      for (uint32_t k = it > (uint32_t)kStages ? it - kStages : 0; k < it; ++k)
        if (!bar_wait(full + 8 * (k % kStages), k / kStages & 1u)) break;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t it = 0, cc = 0;
      bool ok = true;
      for (int t = first; t < p.n_tiles && ok; t += step) {
        const Place pl = place<BN, GROUPED>(p, t);
        const Product& P = *pl.P;
        const int nkb = (P.K + kBlockK - 1) / kBlockK, kb0 = nkb * q / S, kb1 = nkb * (q + 1) / S;
        const uint32_t idesc = instr_desc(p.bf16, P.a_mn, P.b_mn, kTileM, BN);
        // K-major: 8-row groups 1024 bytes apart, 32 bytes per K step.  Rows contiguous: 64-row
        // boxes 8 KB apart, 8-k groups 1024 bytes apart, 16 k rows (2048 bytes) per K step.
        const uint32_t lead_a = P.a_mn ? kBoxBytes : 16, lead_b = P.b_mn ? kBoxBytes : 16;
        const uint64_t step_a = (P.a_mn ? 2048 : 32) >> 4, step_b = (P.b_mn ? 2048 : 32) >> 4;
        for (int ps = 0; ps < P.n_pass && ok; ++ps) {
          for (int k0 = kb0; k0 < kb1 && ok; k0 += P.chunk, ++cc) {
            const int k1 = k0 + P.chunk < kb1 ? k0 + P.chunk : kb1;
            const uint32_t acc = tmem + (cc & 1u) * BN;
            if (!bar_wait(tempty + 8 * (cc & 1u), (cc >> 1 & 1u) ^ 1u)) {
              ok = false;
              break;
            }
            fence_after();
            for (int kb = k0; kb < k1; ++kb, ++it) {
              const uint32_t s = it % kStages;
              if (!bar_wait(full + 8 * s, it / kStages & 1u)) {
                ok = false;
                break;
              }
              fence_after();
              const uint32_t sa = ring + s * stage_bytes(BN);
              const uint64_t da = smem_desc(sa, lead_a, 1024), db = smem_desc(sa + kABytes, lead_b, 1024);
#pragma unroll
              for (int k = 0; k < kBlockK / 16; ++k)
                mma_f16(acc, da + k * step_a, db + k * step_b, idesc, kb > k0 || k > 0);
              mma_commit(empty + 8 * s);
            }
            if (!ok) break;
            mma_commit(tfull + 8 * (cc & 1u));
          }
        }
      }
      if (!ok) {
        atomicOr(p.err, kErrProductWait);
        mma_commit(drain);  // products in flight end before the CTA does
        bar_wait(drain, 0);
      }
    }
    __syncwarp();
  } else {
    constexpr int kHalf = BN / 2;
    const int ew = warp - 2;
    const int quad = warp & 3;            // the TMEM lanes this warp may read
    const int colbase = ew < 4 ? 0 : kHalf;  // warps 2-5 and 6-9 cover each quadrant once
    const int row = quad * 32 + lane;
    uint32_t cc = 0;
    bool ok = true;
    for (int t = first; t < p.n_tiles; t += step) {
      const Place pl = place<BN, GROUPED>(p, t);
      const Product& P = *pl.P;
      const int nkb = (P.K + kBlockK - 1) / kBlockK, kb0 = nkb * q / S, kb1 = nkb * (q + 1) / S;
      float acc[kHalf];
#pragma unroll
      for (int k = 0; k < kHalf; ++k) acc[k] = 0.f;
      for (int ps = 0; ps < P.n_pass; ++ps) {
        const float scale = P.scale[ps];
        for (int k0 = kb0; k0 < kb1; k0 += P.chunk, ++cc) {
          if (ok && !bar_wait(tfull + 8 * (cc & 1u), cc >> 1 & 1u)) ok = false;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) continue;  // the error word is set below; the tile's values are not written
          fence_after();
          const uint32_t at = tmem + (cc & 1u) * BN + colbase + ((uint32_t)(quad * 32) << 16);
          if constexpr (kHalf >= 32) {
#pragma unroll
            for (int c = 0; c < kHalf; c += 32) {
              float v[32];
              tmem_ld32(at + c, v);
#pragma unroll
              for (int k = 0; k < 32; ++k) acc[c + k] += scale * v[k];
            }
          } else {
            float v[16];
            tmem_ld16(at, v);
#pragma unroll
            for (int k = 0; k < 16; ++k) acc[k] += scale * v[k];
          }
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(tempty + 8 * (cc & 1u));
        }
      }
      // the sums to shared memory; the previous tile's have been read
      asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
#pragma unroll
      for (int k = 0; k < kHalf; k += 4)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(staging + (row * kPitch + colbase + k) * 4),
                     "f"(acc[k]), "f"(acc[k + 1]), "f"(acc[k + 2]), "f"(acc[k + 3])
                     : "memory");
      asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
      if (S > 1) break;  // one tile per cluster; its sums are joined below
      if (!ok) continue;
      const int M = P.M, N = P.N;
      if (!P.swap) {
        const bool vec = wide_access<GROUPED>(P, p);
        constexpr int kLanes = BN / 4, kRows = 32 / kLanes;  // lanes on a row, rows at a time
        for (int r = ew * kRows + (vec ? lane / kLanes : 0); r < kTileM; r += kEpiWarps * kRows) {
          if (vec) {
            const int m = pl.row0 + r, c = lane % kLanes * 4, n = pl.col0 + c;
            if (m >= M || n >= N) continue;
            float v[4];
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                         : "r"(staging + (r * kPitch + c) * 4));
            if (n + 4 <= N) {
              emit<4, GROUPED>(P, p, m, n, v);
            } else {
              for (int k = 0; k < 4 && n + k < N; ++k) {
                float u[1] = {v[k]};
                emit<1, GROUPED>(P, p, m, n + k, u);
              }
            }
          } else {
            for (int rr = r; rr < r + kRows; ++rr) {
              const int m = pl.row0 + rr;
              for (int c = lane; c < BN; c += 32) {
                const int n = pl.col0 + c;
                if (m >= M || n >= N) continue;
                float u[1];
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(u[0]) : "r"(staging + (rr * kPitch + c) * 4));
                emit<1, GROUPED>(P, p, m, n, u);
              }
            }
          }
        }
      }
      if (P.swap || pl.mirror) {
        // D(i, j) at output row j, column i: a warp takes 32 rows i, so its stores run along output rows
        for (int u = ew; u < BN; u += kEpiWarps) {
          const int i = (u & 3) * 32 + lane, c = (u >> 2) * 4, n = pl.row0 + i;
          if (n >= M) continue;
          float v[4];
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                       : "r"(staging + (i * kPitch + c) * 4));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (pl.col0 + c + k < N) {
              float w[1] = {v[k]};
              emit<1, GROUPED>(P, p, pl.col0 + c + k, n, w);
            }
        }
      }
    }
    if (!ok && lane == 0) atomicOr(p.err, kErrProductWait);
  }

  if (S > 1) {
    __syncwarp();
    cluster_sync();  // every CTA's sums are in its shared memory
    if (warp >= 2 && first < p.n_tiles) {
      const Place pl = place<BN, GROUPED>(p, first);
      const Product& P = *pl.P;
      const int ew = warp - 2, M = P.M, N = P.N, share = kTileM / S;
      const bool failed = *reinterpret_cast<volatile uint32_t*>(p.err) != 0;
      if (!failed && !P.swap) {
        const bool vec = wide_access<GROUPED>(P, p);
        for (int r = q * share + ew; r < (q + 1) * share; r += kEpiWarps) {
          const int m = pl.row0 + r;
          if (m >= M) continue;
          if (vec) {
            for (int c = lane * 4; c < BN; c += 128) {
              const int n = pl.col0 + c;
              if (n >= N) continue;
              float v[4] = {0.f, 0.f, 0.f, 0.f};
              for (int k = 0; k < S; ++k) {
                const float4 u = ld_peer4(peer_addr(staging + (r * kPitch + c) * 4, k));
                v[0] += u.x, v[1] += u.y, v[2] += u.z, v[3] += u.w;
              }
              if (n + 4 <= N) {
                emit<4, GROUPED>(P, p, m, n, v);
              } else {
                for (int k = 0; k < 4 && n + k < N; ++k) {
                  float u[1] = {v[k]};
                  emit<1, GROUPED>(P, p, m, n + k, u);
                }
              }
            }
          } else {
            for (int c = lane; c < BN; c += 32) {
              const int n = pl.col0 + c;
              if (n >= N) continue;
              float u[1] = {0.f};
              for (int k = 0; k < S; ++k) u[0] += ld_peer(peer_addr(staging + (r * kPitch + c) * 4, k));
              emit<1, GROUPED>(P, p, m, n, u);
            }
          }
        }
      }
      if (!failed && (P.swap || pl.mirror)) {
        for (int u = q * kEpiWarps + ew; u < BN; u += S * kEpiWarps) {
          const int i = (u & 3) * 32 + lane, c = (u >> 2) * 4, n = pl.row0 + i;
          if (n >= M) continue;
          float v[4] = {0.f, 0.f, 0.f, 0.f};
          for (int k = 0; k < S; ++k) {
            const float4 w = ld_peer4(peer_addr(staging + (i * kPitch + c) * 4, k));
            v[0] += w.x, v[1] += w.y, v[2] += w.z, v[3] += w.w;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (pl.col0 + c + k < N) {
              float w[1] = {v[k]};
              emit<1, GROUPED>(P, p, pl.col0 + c + k, n, w);
            }
        }
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while a peer reads its shared memory
  }
  __syncthreads();
  if (warp == 1) {
    fence_after();
    tmem_free(tmem, kCols);
  }
}

template <int BN, bool GROUPED>
cudaError_t launch_one(const ProductLaunch& p, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> sized{0};  // devices whose copy of the kernel may use this much shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !(sized.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(product_kernel<BN, GROUPED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(BN));
    if (e != cudaSuccess) return e;
    if (dev <= 63) sized.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  const int ctas = p.splits > 1 ? p.n_tiles * p.splits : (p.n_tiles < sms ? p.n_tiles : sms);
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(BN);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (p.splits > 1) {
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)p.splits;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, product_kernel<BN, GROUPED>, p);
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

}  // namespace

bool make_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t ld, int box_rows, bool bf16) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {ld * 2};
  const cuuint32_t box[2] = {(cuuint32_t)kBlockK, (cuuint32_t)box_rows};
  const cuuint32_t unit[2] = {1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base),
            dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_product(const ProductLaunch& p, int tile_n, bool grouped, int sms, cudaStream_t stream) {
  if (p.n_tiles <= 0) return cudaSuccess;
  if (grouped) return tile_n == 64 ? launch_one<64, true>(p, sms, stream) : launch_one<128, true>(p, sms, stream);
  if (tile_n == 32) return launch_one<32, false>(p, sms, stream);
  if (tile_n == 64) return launch_one<64, false>(p, sms, stream);
  return launch_one<128, false>(p, sms, stream);
}

}  // namespace ddl
