// product_kernels.cu -- the tensor-core product kernel of the linear layers
// and of the Newton-Schulz steps.
//
//   D(i, j) = sum_pass scale_pass sum_k A_pass(i, k) B_pass(j, k)
//
// on tcgen05 (128 x tile_n tiles on a CTA, 256 x 256 on a CTA pair; accumulators
// in TMEM), then one of the epilogues of product.h.
//
// Roles of a CTA's warps: warp 0 loads operand boxes by TMA into a ring of
// shared-memory stages, warp 1 issues the products, warps 4-11 take the finished
// sums out of TMEM and make the results, warp 2 moves what they read and write,
// a slab of 32 columns at a time, as TMA boxes between memory and four buffers of
// shared memory (rows that TMA cannot address go through one such buffer and are
// written by the warps themselves, along rows).  The two TMEM accumulators
// alternate, so the epilogue of one chunk or tile runs under the products of the
// next.
//
// What bounds it.  256 x 256 x 64 takes a pair 0.28 us at full clocks (about 1.95 GHz, short
// bursts) and 0.34 under the power cap of long runs (1.7 GHz).  In bursts 8192 x 8192 -> 4096
// without an epilogue takes 308 us, the library 300 (1830 TFLOP/s).  A launch adds 4 to 9 us
// and its last epilogue 3 (no activation) to 10 us (GELU, residual, pre-activations):
// 8192 x 4096 -> 4096 takes 156 and 179 us against the library's 141 for the product alone
// (all three 5 % less on another GB300), and the second 189 under the cap.  128 x 128 tiles
// are bound by shared memory (0.31 us for 128 x 128 x 64, half a pair's rate) and are
// taken where pairs would leave SMs idle (choose_layout).  An epilogue slab costs its
// warps 1100 cycles, most of it latency of some 150 instructions, and 800 more with
// GELU: layers with less than 1024 inputs are bound by that (8192 x 512 -> 4096: 41 and
// 72 us).  Two groups of epilogue warps on alternate slabs gained 3 us without and lost
// 4 us with GELU (registers), six stages and two slabs nothing: neither is here.
//
// The tensor core adds with truncation: a long sum of one sign loses about
// half a unit in the last place of each of its K/16 additions.  Results kept in
// binary32 therefore leave the accumulator every `chunk` K blocks and are added
// in registers with rounding to nearest (the first pass's; the sums of lower planes
// are 2^-8 or 2^-11 of those and may stay longer).  16-bit results may stay much
// longer; the forward kernel takes its sums straight from TMEM, and contractions that
// need chunks have a kernel of their own.
//
// A long contraction with few tiles is split over the CTAs of a cluster; each
// leaves its sums in shared memory and the cluster's CTAs add them in rank order
// through distributed shared memory, so results do not depend on timing.  In
// grouped launches a long tile may instead be cut into parts of several workers,
// which are added through memory by the one that comes last.
//
// Every wait is bounded.  One that runs out sets kErrProductWait; the CTA then
// waits (bounded too) for its own loads and products, frees its TMEM and ends.  A
// pair's loads all count on the even CTA's barriers, so it is told how far the odd
// one came, makes up for what either did not ask for, and waits for both's loads
// before either ends (end_loads).

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <type_traits>

#include "activation.cuh"
#include "product.h"
#include "tc_ptx.cuh"

namespace ddl {
namespace {

using namespace tc;

constexpr int kThreads = 384;  // warp 3 only fills the first warpgroup
constexpr int kEpiWarps = 8;
constexpr int kBoxBytes = kBoxRows * kBlockK * 2;
constexpr int kABytes = kTileM * kBlockK * 2;

// This file is compiled twice: as it is, and (product_selftest.cu) with stops that make its waits run out.  Looking for them
// would cost every launch 0.2 us.
#ifdef DDL_PRODUCT_SELFTEST
constexpr bool kSelfTest = true;
#else
constexpr bool kSelfTest = false;
#endif

// What a launch is for; each has its own epilogues (and registers: one that spilled would go to L2 for it, since shared
// memory leaves no L1).
enum : int { kForward, kBackward, kSteps, kForwardLong };
__host__ __device__ constexpr bool is_forward(int mode) { return mode == kForward || mode == kForwardLong; }

// Per CTA: a pair (tile_n 256) splits both operands' rows between its CTAs.
__host__ __device__ constexpr int b_rows(int bn) { return bn == 256 ? 128 : bn; }
__host__ __device__ constexpr int stages(int bn) { return bn >= 128 ? 5 : 6; }
__host__ __device__ constexpr int stage_bytes(int bn) { return kABytes + b_rows(bn) * kBlockK * 2; }
constexpr int kSlab = kSlabCols;
__host__ __device__ constexpr int pitch(int cols) { return cols + 4; }        // floats; rows 4 banks apart
constexpr int kPlaneBytes = kTileM * kSlab * 2;  // a slab of 16 bits
constexpr int kSlabBytes = 2 * kPlaneBytes;      // what a box epilogue keeps of a slab: two planes, or binary32
constexpr int kBufs = 4;                         // slabs on their way in, in work and on their way out
__host__ __device__ constexpr int smem_bytes(int bn) {
  return 1024 + stages(bn) * stage_bytes(bn) + (bn >= 128 ? kBufs * kSlabBytes : kTileM * pitch(kSlab) * 4);
}

// -- element access -------------------------------------------------------------

template <int V>
__device__ __forceinline__ void load16(const void* base, int64_t at, int type, float (&v)[V]) {
  const uint16_t* p = static_cast<const uint16_t*>(base) + at;
  if constexpr (V == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = from16x2(u.x, type), b = from16x2(u.y, type);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  } else {
    v[0] = from16(*p, type);
  }
}

template <int V>
__device__ __forceinline__ void store16(void* base, int64_t at, int type, const float (&v)[V]) {
  uint16_t* p = static_cast<uint16_t*>(base) + at;
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(to16x2(v[0], v[1], type), to16x2(v[2], v[3], type));
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

// -- epilogues ---------------------------------------------------------------------

template <int V, int R, int ACT>
__device__ __forceinline__ void activate_all(float (&v)[R][V]) {
  constexpr int N = (R * V + 1) / 2 * 2;
  float u[N] = {};
#pragma unroll
  for (int k = 0; k < R * V; ++k) u[k] = v[k / V][k % V];
  activate<ACT>(u);
#pragma unroll
  for (int k = 0; k < R * V; ++k) v[k / V][k % V] = u[k];
}

template <int V, int R, int TYPE>
__device__ __forceinline__ void emit_linear(const Product& P, const int (&m)[R], const bool (&in)[R], int n,
                                            float (&v)[R][V]) {
  float t[V], add[R][V];
  if (P.add) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (in[i]) load16(P.add, (int64_t)m[i] * P.ld_add + n, TYPE, add[i]);
  }
  if (P.bias) {
    load16(P.bias, n, TYPE, t);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) v[i][k] += t[k];
  }
  if (P.z) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (in[i]) store16(P.z, (int64_t)m[i] * P.ldz + n, TYPE, v[i]);
  }
  switch (P.act) {
    case kActRelu: activate_all<V, R, kActRelu>(v); break;
    case kActGelu: activate_all<V, R, kActGelu>(v); break;
    case kActSilu: activate_all<V, R, kActSilu>(v); break;
    default: break;
  }
  if (P.add) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) v[i][k] += add[i][k];
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (in[i]) store16(P.out, (int64_t)m[i] * P.ldo + n, TYPE, v[i]);
}

// V values of D in each of R rows of a linear layer's result: rows m[i] of the output (where in[i]), columns n...
// Every load of the R rows is issued before the first is used.
template <int V, int R, int MODE>
__device__ __forceinline__ void emit(const Product& P, const int (&m)[R], const bool (&in)[R], int n, float (&v)[R][V]) {
  if constexpr (is_forward(MODE)) {
    // one branch on the type and one on the activation for all R x V values
    if (P.type == kBF16)
      emit_linear<V, R, kBF16>(P, m, in, n, v);
    else
      emit_linear<V, R, kF16>(P, m, in, n, v);
  } else {
    if (P.accumulate) {
      float t[R][V];
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (in[i]) load_any(P.out, (int64_t)m[i] * P.ldo + n, P.out_type, t[i]);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][k] += t[i][k];
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (in[i]) store_any(P.out, (int64_t)m[i] * P.ldo + n, P.out_type, v[i]);
  }
}

// One element at the edge of the wide path, out of line so that the code around it stays small.  `P` is the launch's own
// record.
template <int MODE>
__device__ __noinline__ void emit_one(const Product* P, int m, int n, float x) {
  const int mm[1] = {m};
  const bool in[1] = {true};
  float v[1][1] = {{x}};
  emit<1, 1, MODE>(*P, mm, in, n, v);
}

// The epilogue warps' own barrier.
__device__ __forceinline__ void bar_sync_epilogue() {
  asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
}

// What the loops over a tile's contraction read of its product, in registers: a load from the product's own memory
// would be repeated after every wait.
struct Shape {
  int kb0, kb1, chunk0, chunk1, n_pass, a_mn, b_mn;
  float scale0, scale1, scale2;
  // part `part` of `parts` of K blocks [k0, k1)
  __device__ __forceinline__ Shape(const Product& P, int k0, int k1, int part, int parts)
      : chunk0(P.chunk[0]),
        chunk1(P.chunk[1]),
        n_pass(P.n_pass),
        a_mn(P.a_mn),
        b_mn(P.b_mn),
        scale0(P.scale[0]),
        scale1(P.scale[1]),
        scale2(P.scale[2]) {
    kb0 = k0 + (k1 - k0) * part / parts;
    kb1 = k0 + (k1 - k0) * (part + 1) / parts;
  }
  __device__ __forceinline__ int chunk(int pass) const { return pass ? chunk1 : chunk0; }
  __device__ __forceinline__ float scale(int pass) const { return pass == 0 ? scale0 : pass == 1 ? scale1 : scale2; }
};

// A place in a ring, and how often that was gone round (modulo 2^32).
struct Slot {
  uint32_t s = 0, lap = 0;
  __device__ __forceinline__ uint32_t parity() const { return lap & 1u; }
  template <int STAGES>
  __device__ __forceinline__ void next() {
    if (++s == STAGES) {
      s = 0;
      ++lap;
    }
  }
  // uses so far, modulo 2^32
  template <int STAGES>
  __device__ __forceinline__ uint32_t uses() const {
    return lap * STAGES + s;
  }
};

// After a pair gave up: waits (bounded) on the even CTA's barriers for the loads of both.  The even one would have gone on
// at `at`; the odd one asked for `more` K blocks more than it (or fewer: < 0).  A barrier's phase ends with the even CTA's
// arrival, which tells it of both halves, and their bytes; of a block that only one of them asked for the other's part is
// made up here.  They differ by at most STAGES blocks, since a slot is not asked for again before the products of its last
// use are done.
template <int STAGES>
__device__ __forceinline__ void end_loads(uint32_t full, uint32_t half, Slot at, int more, uint64_t limit) {
  const int most = more > 0 ? more : 0;
  // the last use of every slot, counted from the even CTA's next one; of a slot without any, the lap before the first, which
  // counts as done
  for (int n = most - STAGES; n < most; ++n) {
    const int back = (int)at.s + n;  // -STAGES .. 2 STAGES - 2
    const int slot = (back + STAGES) % STAGES, laps = (back + STAGES) / STAGES - 1;
    const uint32_t bar = full + 8 * slot;
    if (n >= more) bar_complete(bar, half);
    if (n >= 0) bar_expect(bar, half);
    if (!bar_wait(bar, (at.lap + laps) & 1u, limit)) break;
  }
}

// Makes a tensor map that the host wrote into device memory usable by this thread's TMA operations.
__device__ __forceinline__ void acquire_map(const CUtensorMap* map) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(map) : "memory");
}

struct Place {
  const Product* P;
  int row0, col0, mirror;
  int k0, k1;
  int part, parts, slot, count;
  int next;  // the worker's next tile
};

template <int BN, int MODE>
__device__ __forceinline__ Place place(const ProductLaunch& p, int t, int step) {
  constexpr int BM = BN == 256 ? 2 * kTileM : kTileM;
  if constexpr (MODE == kSteps) {
    const int4* tile = reinterpret_cast<const int4*>(p.g_tiles + t);
    const int4 u = __ldg(tile), k = __ldg(tile + 1), w = __ldg(tile + 2);
    return {p.g_products + u.x, u.y * BM, u.z * BN, u.w, k.x, k.y, k.z, k.w, w.x, w.y, w.z};
  } else {
    const int next = t + step;
    int k = 0;
    if (MODE == kBackward && t >= p.inl_tiles[0]) {  // forward launches have one product
      k = 1;
      t -= p.inl_tiles[0];
    }
    const Product* P = &p.inl[k];
    // bands of 16 tile rows, column by column, so that CTAs in flight share operands in L2
    const int rows = (P->M + BM - 1) / BM, cols = (P->N + BN - 1) / BN;
    const int band = t / (16 * cols), first = band * 16;
    const int height = rows - first < 16 ? rows - first : 16;
    const int in = t - band * 16 * cols;
    return {P, (first + in % height) * BM, in / height * BN, 0, 0, (P->K + kBlockK - 1) / kBlockK, 0, 1, 0, 0, next};
  }
}

// Where a tile's sums lie between the epilogue's two halves: this CTA's shared memory, or the shared memories of a
// cluster whose CTAs each hold part of every sum.
struct OwnSums {
  uint32_t base;
  __device__ __forceinline__ float one(uint32_t at) const { return ld_shared(base + at); }
  __device__ __forceinline__ void four(uint32_t at, float (&v)[4]) const { ld_shared4(base + at, v); }
};
struct ClusterSums {
  uint32_t base;
  int parts;         // 2, 4 or 8
  int first, apart;  // their CTAs' ranks
  template <int PARTS>
  __device__ __forceinline__ void add4(uint32_t at, float (&v)[4]) const {
    float4 u[PARTS];
#pragma unroll
    for (int k = 0; k < PARTS; ++k) u[k] = ld_peer4(peer_addr(base + at, first + k * apart));
#pragma unroll
    for (int k = 0; k < PARTS; ++k) v[0] += u[k].x, v[1] += u[k].y, v[2] += u[k].z, v[3] += u[k].w;
  }
  __device__ __forceinline__ float one(uint32_t at) const {
    float v = 0.f;
    for (int k = 0; k < parts; ++k) v += ld_peer(peer_addr(base + at, first + k * apart));
    return v;
  }
  __device__ __forceinline__ void four(uint32_t at, float (&v)[4]) const {
    v[0] = v[1] = v[2] = v[3] = 0.f;
    if (parts == 2)
      add4<2>(at, v);
    else if (parts == 4)
      add4<4>(at, v);
    else
      add4<8>(at, v);
  }
};

// Writes rows [r0, r1) of 128 x COLS sums that begin at D(row0, col0), along rows of D.  `from` is the record that P is a
// copy of.
template <int COLS, int MODE, bool WHOLE, class Sums>
__device__ __forceinline__ void write_rows_wide(const Product& P, const Product* from, int row0, int col0, int lane, int ew,
                                                int r0, int r1, const Sums sums) {
  constexpr int kPitch = pitch(COLS), kBatch = 4;
  constexpr int kLanes = COLS / 4 < 32 ? COLS / 4 : 32, kRows = 32 / kLanes;  // lanes on a row, rows at a time
  for (int c = lane % kLanes * 4; c < COLS; c += kLanes * 4) {
    const int n = col0 + c;
    if (!WHOLE && n >= P.N) continue;
#pragma unroll 1
    for (int rr = r0 + ew * kRows + lane / kLanes; rr < r1; rr += kEpiWarps * kRows * kBatch) {
      int m[kBatch];
      bool in[kBatch];
      float v[kBatch][4];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = rr + i * kEpiWarps * kRows;
        m[i] = row0 + r;
        in[i] = WHOLE || (r < r1 && m[i] < P.M);
        if (in[i]) sums.four((r * kPitch + c) * 4, v[i]);
      }
      if (WHOLE || n + 4 <= P.N) {
        emit<4, kBatch, MODE>(P, m, in, n, v);
      } else {
#pragma unroll 1
        for (int k = 0; n + k < P.N; ++k)
#pragma unroll 1
          for (int i = 0; i < kBatch; ++i) {
            const int r = rr + i * kEpiWarps * kRows;
            if (r < r1 && row0 + r < P.M) emit_one<MODE>(from, row0 + r, n + k, sums.one((r * kPitch + c + k) * 4));
          }
      }
    }
  }
}

template <int COLS, int MODE, class Sums>
__device__ __forceinline__ void write_rows(const Product& P, const Product* from, int row0, int col0, int lane, int ew, int r0,
                                           int r1, const Sums sums) {
  constexpr int kStride = kEpiWarps * 4 * (COLS / 4 < 32 ? 128 / COLS : 1);  // rows a pass of all warps covers
  if (P.vec) {
    // tiles that lie wholly inside need no predicate anywhere
    if (row0 + r1 <= P.M && col0 + COLS <= P.N && (r1 - r0) % kStride == 0)
      write_rows_wide<COLS, MODE, true>(P, from, row0, col0, lane, ew, r0, r1, sums);
    else
      write_rows_wide<COLS, MODE, false>(P, from, row0, col0, lane, ew, r0, r1, sums);
  } else {  // rows at any alignment: a warp along a row, element by element, four rows at a time
#pragma unroll 1
    for (int c = lane; c < COLS; c += 32) {
      if (col0 + c >= P.N) break;
#pragma unroll 1
      for (int rr = r0 + ew; rr < r1; rr += kEpiWarps * 4) {
        int m[4];
        bool in[4];
        float v[4][1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = rr + i * kEpiWarps;
          m[i] = row0 + r;
          in[i] = r < r1 && m[i] < P.M;
          v[i][0] = in[i] ? sums.one((r * pitch(COLS) + c) * 4) : 0.f;
        }
        emit<1, 4, MODE>(P, m, in, col0 + c, v);
      }
    }
  }
}

// Writes rows [r0, r0 + rows) of the sums with D(i, j) at output row j, column i: neighbouring lanes take neighbouring
// rows i, so that stores run along output rows, and four columns j.  rows is 16, 32, 64 or 128.
template <int COLS, int MODE, class Sums>
__device__ __forceinline__ void write_transposed(const Product& P, int row0, int col0, int thread, int r0, int rows,
                                                 const Sums sums) {
  constexpr int kPitch = pitch(COLS);
#pragma unroll 1
  for (int u = thread; u < rows * (COLS / 4); u += kEpiWarps * 32) {
    const int i = r0 + u % rows, c = u / rows * 4, n = row0 + i;
    if (n >= P.M || col0 + c >= P.N) continue;
    float v[4];
    sums.four((i * kPitch + c) * 4, v);
    int m[4];
    bool in[4];
    float w[4][1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      m[k] = col0 + c + k;
      in[k] = m[k] < P.N;
      w[k][0] = v[k];
    }
    emit<1, 4, MODE>(P, m, in, n, w);
  }
}

// -- box epilogues ------------------------------------------------------------------
//
// 32 columns of a tile at a time.  A thread has 16 columns of one row; what it reads (residual, old output, C's
// planes) TMA has put into a slab of shared memory, the results replace it there in place, and TMA stores the slab.
// A box that the matrix's edge cuts is stored in whole 16-byte pieces, so a caller's rows end on one where boxes are used.
// A plane's rows are 64 bytes with the 64-byte swizzle: 16-byte piece c of row r lies at piece c ^ (r / 2 & 3).  Binary32
// rows are 128 bytes with the 128-byte swizzle: at piece c ^ (r & 7).

__device__ __forceinline__ uint32_t piece(uint32_t plane, int row, int c) {
  return plane + row * 64 + ((c ^ (row >> 1 & 3)) << 4);
}
__device__ __forceinline__ uint32_t piece32(uint32_t slab, int row, int c) {
  return slab + row * 128 + ((c ^ (row & 7)) << 4);
}

__device__ __forceinline__ void unpack8(uint4 u, int type, float (&v)[8]) {
  const float2 a = from16x2(u.x, type), b = from16x2(u.y, type), c = from16x2(u.z, type), d = from16x2(u.w, type);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y, v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
}

__device__ __forceinline__ uint4 pack8(const float* v, int type) {
  return make_uint4(to16x2(v[0], v[1], type), to16x2(v[2], v[3], type), to16x2(v[4], v[5], type), to16x2(v[6], v[7], type));
}

// The planes of 8 values x kPlaneScale.
__device__ __forceinline__ void split8(const float* x, uint4* hi, uint4* lo) {
  float h[8], l[8];
  *hi = pack8(x, kF16);
  unpack8(*hi, kF16, h);
#pragma unroll
  for (int k = 0; k < 8; ++k) l[k] = x[k] - h[k];
  *lo = pack8(l, kF16);
}

// Stores 8 columns n.. of the warp's 32 rows at their mirror images.  Lanes 2k and 2k + 1 trade halves, so that each has
// two neighbouring rows of one column, and 16 lanes write 64 bytes of an image row.  row0 + row is even on even lanes; the
// row after the last, if a lane pair has one, falls into the padding.
__device__ __forceinline__ void store_mirror8(uint16_t* plane, int64_t ld, uint4 u, int row, int rows, int n, int cols,
                                              int lane) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  const int odd = lane & 1;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, w[k], 1);
    const uint32_t pair = odd ? __byte_perm(other, w[k], 0x7632) : __byte_perm(w[k], other, 0x5410);
    const int c = n + 2 * k + odd, r = row - odd;
    if (r < rows && c < cols) *reinterpret_cast<uint32_t*>(plane + (int64_t)c * ld + r) = pair;
  }
}

template <int TYPE, int ACT>
__device__ __forceinline__ void slab_linear(const Product& P, float* v, const uint4 (&bias)[2], uint32_t buf, int row,
                                            int half) {
  const uint32_t at[2] = {piece(buf, row, 2 * half), piece(buf, row, 2 * half + 1)};
  uint4 add[2];
  if (P.in0 >= 0) add[0] = ld_shared16(at[0]), add[1] = ld_shared16(at[1]);
  float u[16];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    float t[8];
    unpack8(bias[g], TYPE, t);
#pragma unroll
    for (int k = 0; k < 8; ++k) u[8 * g + k] = v[8 * g + k] + t[k];
  }
  if (P.out1 >= 0) {
    st_shared16(at[0] + kPlaneBytes, pack8(u, TYPE));
    st_shared16(at[1] + kPlaneBytes, pack8(u + 8, TYPE));
  }
  activate<ACT>(u);
  if (P.in0 >= 0) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      float t[8];
      unpack8(add[g], TYPE, t);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[8 * g + k] += t[k];
    }
  }
  st_shared16(at[0], pack8(u, TYPE));
  st_shared16(at[1], pack8(u + 8, TYPE));
}

template <int TYPE>
__device__ __forceinline__ void slab_linear_act(const Product& P, float* v, const uint4 (&bias)[2], uint32_t buf, int row,
                                                int half) {
  switch (P.act) {
    case kActRelu: slab_linear<TYPE, kActRelu>(P, v, bias, buf, row, half); break;
    case kActGelu: slab_linear<TYPE, kActGelu>(P, v, bias, buf, row, half); break;
    case kActSilu: slab_linear<TYPE, kActSilu>(P, v, bias, buf, row, half); break;
    default: slab_linear<TYPE, kActNone>(P, v, bias, buf, row, half); break;
  }
}

// 16 columns n.. of the bias (zeros without one, or outside: rows are whole pieces).
__device__ __forceinline__ void load_bias(const Product& P, int n, uint4 (&bias)[2]) {
#pragma unroll
  for (int g = 0; g < 2; ++g)
    bias[g] = P.bias && n + 8 * g < P.N ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.bias) + n + 8 * g))
                                        : make_uint4(0, 0, 0, 0);
}

template <int MODE>
__device__ __forceinline__ void slab_values(const Product& P, const ProductLaunch& p, float* v, const uint4 (&bias)[2],
                                            uint32_t buf, int row, int half, int row0, int n0, bool mirror) {
  if constexpr (MODE == kSteps) {
    // v is D in binary32, C's planes hold kPlaneScale times its values, as the result's will
    const float cc = P.epi == kEpiPoly ? p.cb : p.ca, cd = (P.epi == kEpiPoly ? p.cc : 1.f) * kPlaneScale;
    const uint32_t at[2] = {piece(buf, row, 2 * half), piece(buf, row, 2 * half + 1)};
    if (P.in0 >= 0) {
      uint4 h[2], l[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) h[g] = ld_shared16(at[g]), l[g] = ld_shared16(at[g] + kPlaneBytes);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float a[8], b[8];
        unpack8(h[g], kF16, a);
        unpack8(l[g], kF16, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[8 * g + k] = cd * v[8 * g + k] + cc * (a[k] + b[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] *= kPlaneScale;
    }
    uint4 hi[2], lo[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) split8(v + 8 * g, &hi[g], &lo[g]);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      st_shared16(at[g], hi[g]);
      st_shared16(at[g] + kPlaneBytes, lo[g]);
    }
    if (mirror) {  // D(i, j) also at (j, i): the warp's 32 rows i lie side by side there
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        store_mirror8(P.p_hi, P.ldp, hi[g], row0 + row, P.M, n0 + 8 * g, P.N, row & 31);
        store_mirror8(P.p_lo, P.ldp, lo[g], row0 + row, P.M, n0 + 8 * g, P.N, row & 31);
      }
    }
  } else if constexpr (is_forward(MODE)) {
    if (P.type == kBF16)
      slab_linear_act<kBF16>(P, v, bias, buf, row, half);
    else
      slab_linear_act<kF16>(P, v, bias, buf, row, half);
  } else if (P.out_type == kF32) {
    float t[4][4];
    if (P.in0 >= 0) {
#pragma unroll
      for (int g = 0; g < 4; ++g) ld_shared4(piece32(buf, row, 4 * half + g), t[g]);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] += t[k >> 2][k & 3];
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) st_shared4(piece32(buf, row, 4 * half + g), v + 4 * g);
  } else {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint32_t at = piece(buf, row, 2 * half + g);
      float* x = v + 8 * g;
      if (P.in0 >= 0) {
        float t[8];
        unpack8(ld_shared16(at), P.out_type, t);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] += t[k];
      }
      st_shared16(at, pack8(x, P.out_type));
    }
  }
}

__device__ __forceinline__ void unpack4(uint2 u, float (&v)[4]) {
  const float2 a = from16x2(u.x, kF16), b = from16x2(u.y, kF16);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

// The planes of 4 values x kPlaneScale.
__device__ __forceinline__ void split4(const float (&x)[4], uint2* hi, uint2* lo) {
  float h[4];
  *hi = make_uint2(to16x2(x[0], x[1], kF16), to16x2(x[2], x[3], kF16));
  unpack4(*hi, h);
  *lo = make_uint2(to16x2(x[0] - h[0], x[1] - h[1], kF16), to16x2(x[2] - h[2], x[3] - h[3], kF16));
}

// Where the contraction was split: finishes rows [r0, r0 + rows) of the BN columns at D(row0, col0), along rows of the
// planes (padded to 8 columns, so that a group of 4 that begins inside the matrix is whole).  back: the finished values,
// x kPlaneScale, also replace the sums in this CTA's shared memory.
template <int BN>
__device__ __forceinline__ void joined_rows(const Product& P, const ProductLaunch& p, const ClusterSums sums, int row0,
                                            int col0, int r0, int rows, int ew, int lane, bool back) {
  constexpr int kBatch = 4;
  const float cc = P.epi == kEpiPoly ? p.cb : p.ca, cd = (P.epi == kEpiPoly ? p.cc : 1.f) * kPlaneScale;
#pragma unroll 1
  for (int c = lane * 4; c < BN; c += 128) {
    const int n = col0 + c;
    if (n >= P.N) continue;
#pragma unroll 1
    for (int rr = ew; rr < rows; rr += kEpiWarps * kBatch) {
      uint2 h[kBatch], l[kBatch];
      float v[kBatch][4];
      bool in[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int m = row0 + r0 + rr + i * kEpiWarps;
        in[i] = rr + i * kEpiWarps < rows && m < P.M;
        if (in[i] && P.epi != kEpiGram) {
          h[i] = *reinterpret_cast<const uint2*>(P.c_hi + (int64_t)m * P.ldc + n);
          l[i] = *reinterpret_cast<const uint2*>(P.c_lo + (int64_t)m * P.ldc + n);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (in[i]) sums.four(((r0 + rr + i * kEpiWarps) * pitch(BN) + c) * 4, v[i]);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (!in[i]) continue;
        if (P.epi != kEpiGram) {
          float a[4], b[4];
          unpack4(h[i], a);
          unpack4(l[i], b);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[i][k] = cd * v[i][k] + cc * (a[k] + b[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) v[i][k] *= kPlaneScale;
        }
        uint2 hi, lo;
        split4(v[i], &hi, &lo);
        const int64_t to = (int64_t)(row0 + r0 + rr + i * kEpiWarps) * P.ldp + n;
        *reinterpret_cast<uint2*>(P.p_hi + to) = hi;
        *reinterpret_cast<uint2*>(P.p_lo + to) = lo;
        if (back) st_shared4(sums.base + ((r0 + rr + i * kEpiWarps) * pitch(BN) + c) * 4, v[i]);
      }
    }
  }
}

// The mirror image of what joined_rows finished: neighbouring lanes take neighbouring rows of D, so that the stores run
// along the image's rows.  rows is 16, 32 or 64.
template <int BN>
__device__ __forceinline__ void joined_mirror(const Product& P, uint32_t base, int row0, int col0, int r0, int rows,
                                              int thread) {
#pragma unroll 2
  for (int u = thread; u < rows * (BN / 4); u += kEpiWarps * 32) {
    const int i = r0 + u % rows, c = u / rows * 4, n = row0 + i;
    if (n >= P.M || col0 + c >= P.N) continue;
    float v[4];
    ld_shared4(base + (i * pitch(BN) + c) * 4, v);
    uint2 hi, lo;
    split4(v, &hi, &lo);
    const uint32_t h[2] = {hi.x, hi.y}, l[2] = {lo.x, lo.y};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (col0 + c + k >= P.N) continue;
      const int64_t to = (int64_t)(col0 + c + k) * P.ldp + n;
      P.p_hi[to] = (uint16_t)(h[k >> 1] >> (k & 1) * 16);
      P.p_lo[to] = (uint16_t)(l[k >> 1] >> (k & 1) * 16);
    }
  }
}

// One walk over the slabs of a CTA's tiles: the warp that moves the boxes has two, for what it prepares and for what
// it stores.
template <int BN, int MODE>
struct Slabs {
  int t, end, step, sl, n_sl;
  int row0, col0, following;
  int in0, in1, out0, out1, f32, rows;
  __device__ __forceinline__ Slabs(const ProductLaunch& p, int first, int last, int by)
      : t(first), end(last), step(by), sl(0) {
    load(p);
  }
  __device__ __forceinline__ void load(const ProductLaunch& p) {
    if (t >= end) return;
    const Place pl = place<BN, MODE>(p, t, step);
    row0 = pl.row0, col0 = pl.col0, following = pl.next;
    const Product& P = is_forward(MODE) ? p.inl[0] : *pl.P;
    in0 = P.in0, in1 = P.in1, out0 = P.out0, out1 = P.out1;
    f32 = MODE == kBackward && P.out_type == kF32;
    rows = P.M;
    if constexpr (MODE == kSteps) {  // of the walks, the one that fills and the one that stores each use their own
      if (in0 >= 0) acquire_map(p.g_maps + in0);
      if (in1 >= 0) acquire_map(p.g_maps + in1);
      acquire_map(p.g_maps + out0);
      acquire_map(p.g_maps + out1);
    }
    const int left = (P.N - pl.col0 + kSlab - 1) / kSlab;
    n_sl = left < BN / kSlab ? left : BN / kSlab;
  }
  __device__ __forceinline__ bool more() const { return t < end; }
  __device__ __forceinline__ void next(const ProductLaunch& p) {
    if (++sl < n_sl) return;
    sl = 0;
    t = following;
    load(p);
  }
};

// BN 256: a pair of CTAs makes a 256 x 256 tile, each CTA 128 of its rows, from one stream of products that the even
// CTA issues for both.
template <int BN, int MODE>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ ProductLaunch p) {
  constexpr bool PAIR = BN == 256;
  constexpr bool DIRECT = MODE == kForward;  // one chunk: sums go from TMEM to the epilogue
  constexpr int kStages = stages(BN);
  constexpr uint32_t kCols = 2 * BN;
  constexpr int kSlabPitch = pitch(kSlab), kHalf = kSlab / 2, kSlabs = BN / kSlab;
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t bars[2 * kStages + 5 + 2 * kBufs];
  __shared__ uint32_t tmem_slot;
  __shared__ uint32_t load_slot, load_lap;  // PAIR: where this CTA's loads would have gone on
  __shared__ uint32_t broken, drains;       // PAIR: a CTA of the cluster gave up; this pair's products were cut short
  __shared__ int joins;                  // this CTA's part of a tile was the last: it finishes the tile
  __shared__ volatile int empty_slab[kBufs];  // a slab of a part whose tile another CTA finishes
  const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t staging = ring + kStages * stage_bytes(BN);
  const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages, tempty = tfull + 16,
                 drain = tempty + 16, ready = drain + 8, written = ready + 8 * kBufs;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(full + 8 * s, 1);
      bar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      bar_init(tfull + 8 * b, 1);
      bar_init(tempty + 8 * b, PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    for (int b = 0; b < kBufs; ++b) {
      bar_init(ready + 8 * b, 1);
      bar_init(written + 8 * b, kEpiWarps);
    }
    bar_init(drain, 1);
    broken = drains = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    tmem_alloc<PAIR>(smem_u32(&tmem_slot), kCols);
    fence_before();
  }
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the peer's barriers exist
  fence_after();
  const uint32_t tmem = tmem_slot;
  griddep_launch();
  // Every role reads its first tile's records (the handle's own, or this launch's) before it waits for the kernel
  // before this one, whose results only then may be touched.

  // a cluster has S parts of a tile's contraction, each a CTA's or a pair's
  const int S = p.splits;
  const int rank = PAIR || S > 1 ? (int)cluster_rank() : 0;
  const int odd = PAIR ? rank & 1 : 0, lead = rank - odd;
  const int q = PAIR ? rank >> 1 : rank;
  const int ctas = PAIR ? 2 * S : S;
  // this worker's tiles: a list, or every step-th
  const int first = blockIdx.x / ctas, step = gridDim.x / ctas, end = MODE == kSteps ? kNoTile : p.n_tiles;
  const int my_rows = odd * kTileM;  // this CTA's part of the tile's rows
  const CUtensorMap* maps = MODE == kSteps ? p.g_maps : p.maps;
  const uint64_t limit = kSelfTest ? p.give_up.wait_ns : kWaitLimitNs;

  // The epilogue's sums want registers: 384 threads of 168 become 128 of 56 and 256 of 224 (64,512 either way).
  __syncwarp();
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      Slot at;
      bool ok = true;
      for (int t = first, next; t < end && ok; t = next) {
        const Place pl = place<BN, MODE>(p, t, step);
        next = pl.next;
        const Product& P = *pl.P;
        const Shape sh(P, pl.k0, pl.k1, q, S);
        const CUtensorMap *ma0 = maps + P.a[0], *ma1 = maps + P.a[1], *ma2 = maps + P.a[2];
        const CUtensorMap *mb0 = maps + P.b[0], *mb1 = maps + P.b[1], *mb2 = maps + P.b[2];
        if constexpr (MODE == kSteps) {
          // written by the host before this launch; of three passes the first two share A, the outer two B
          acquire_map(ma0);
          acquire_map(ma2);
          acquire_map(mb0);
          acquire_map(mb1);
        }
        if (t == first) griddep_wait();
        for (int ps = 0; ps < sh.n_pass && ok; ++ps) {
          const CUtensorMap* ma = ps == 0 ? ma0 : ps == 1 ? ma1 : ma2;
          const CUtensorMap* mb = ps == 0 ? mb0 : ps == 1 ? mb1 : mb2;
          for (int kb = sh.kb0; kb < sh.kb1; ++kb, at.next<kStages>()) {
            const uint32_t s = at.s;
            const bool stop = kSelfTest && at.uses<kStages>() == p.give_up.loads[odd];
            if (stop || !bar_wait(empty + 8 * s, at.parity() ^ 1u, limit)) {
              ok = false;
              break;
            }
            const uint32_t sa = ring + s * stage_bytes(BN), sb = sa + kABytes;
            uint32_t bar = full + 8 * s;
            if constexpr (PAIR) {  // both CTAs' loads count on the even one's barrier
              if (!odd)
                bar_expect(bar, 2 * stage_bytes(BN));
              else
                bar = peer_addr(bar, lead);
            } else {
              bar_expect(bar, stage_bytes(BN));
            }
#pragma unroll
            for (int h = 0; h < (is_forward(MODE) ? 1 : kTileM / kBoxRows); ++h) {
              const int row = pl.row0 + my_rows + h * kBoxRows;
              const int x = sh.a_mn ? row : kb * kBlockK, y = sh.a_mn ? kb * kBlockK : row;
              if constexpr (PAIR)
                tma_box_pair(sa + h * kBoxBytes, ma, bar, x, y);
              else
                tma_box(sa + h * kBoxBytes, ma, bar, x, y);
            }
#pragma unroll
            for (int h = 0; h < (is_forward(MODE) ? 1 : (b_rows(BN) + kBoxRows - 1) / kBoxRows); ++h) {
              const int row = pl.col0 + my_rows + h * kBoxRows;
              const int x = sh.b_mn ? row : kb * kBlockK, y = sh.b_mn ? kb * kBlockK : row;
              if constexpr (PAIR)
                tma_box_pair(sb + h * kBoxBytes, mb, bar, x, y);
              else
                tma_box(sb + h * kBoxBytes, mb, bar, x, y);
            }
          }
        }
      }
      if (!ok) atomicOr(p.err, kErrProductWait);
      // Loads in flight end before the CTA does.
      if constexpr (PAIR) {
        load_slot = at.s, load_lap = at.lap;  // see the kernel's end
        if (!ok)
          for (int r = 0; r < 2 * p.splits; ++r) st_peer(peer_addr(smem_u32(&broken), r), 1);
      } else {
        // every slot's last use, the oldest first (one without any counts as done)
        for (int k = 0; k < kStages; ++k, at.next<kStages>())
          if (!bar_wait(full + 8 * at.s, at.parity() ^ 1u, limit)) break;
      }
    }
    if (warp == 1 && lane == 0 && !odd) {
      uint32_t cc = 0;
      Slot at;
      bool ok = true;
      griddep_wait();
      for (int t = first, next; t < end && ok; t = next) {
        const Place pl = place<BN, MODE>(p, t, step);
        next = pl.next;
        const Shape sh(*pl.P, pl.k0, pl.k1, q, S);
        const uint32_t idesc = instr_desc(p.bf16, sh.a_mn, sh.b_mn, PAIR ? 2 * kTileM : kTileM, BN);
        // K-major: 8-row groups 1024 bytes apart, 32 bytes per K step.  Rows contiguous: 64-row
        // boxes 8 KB apart, 8-k groups 1024 bytes apart, 16 k rows (2048 bytes) per K step.
        const uint64_t desc_a = smem_desc(ring, sh.a_mn ? kBoxBytes : 16, 1024);
        const uint64_t desc_b = smem_desc(ring + kABytes, sh.b_mn ? kBoxBytes : 16, 1024);
        const uint64_t step_a = (sh.a_mn ? 2048 : 32) >> 4, step_b = (sh.b_mn ? 2048 : 32) >> 4;
        for (int ps = 0; ps < sh.n_pass && ok; ++ps) {
          const int chunk = sh.chunk(ps);
          for (int k0 = sh.kb0; k0 < sh.kb1 && ok; k0 += chunk, ++cc) {
            const int k1 = k0 + chunk < sh.kb1 ? k0 + chunk : sh.kb1;
            const uint32_t acc = tmem + (cc & 1u) * BN;
            const bool stop = kSelfTest && cc == p.give_up.products;
            if (stop || !bar_wait(tempty + 8 * (cc & 1u), (cc >> 1 & 1u) ^ 1u, limit)) {
              ok = false;
              break;
            }
            fence_after();
            for (int kb = k0; kb < k1; ++kb, at.next<kStages>()) {
              const uint32_t s = at.s;
              if (!bar_wait(full + 8 * s, at.parity(), limit)) {
                ok = false;
                break;
              }
              fence_after();
              const uint64_t da = desc_a + s * (stage_bytes(BN) >> 4), db = desc_b + s * (stage_bytes(BN) >> 4);
#pragma unroll
              for (int k = 0; k < kBlockK / 16; ++k)
                mma_f16<PAIR>(acc, da + k * step_a, db + k * step_b, idesc, kb > k0 || k > 0);
              mma_commit<PAIR>(empty + 8 * s, lead);
            }
            if (!ok) break;
            mma_commit<PAIR>(tfull + 8 * (cc & 1u), lead);
          }
        }
      }
      if (!ok) {
        atomicOr(p.err, kErrProductWait);
        mma_commit<PAIR>(drain, lead);  // products in flight end before the CTA does
        bar_wait(drain, 0, limit);
        if constexpr (PAIR) {
          for (int r = lead; r < lead + 2; ++r) st_peer(peer_addr(smem_u32(&drains), r), 1);
          for (int r = 0; r < 2 * p.splits; ++r) st_peer(peer_addr(smem_u32(&broken), r), 1);
        }
      }
    }
    if constexpr (BN >= 128) {
      if (warp == 2 && lane == 0 && p.boxes) {
        // The slabs of this CTA's tiles take the four buffers in turn: one is filled (or declared free) here, worked on by
        // the epilogue warps, stored here, and can be filled again once the store has read it.  Three are filled ahead,
        // which leaves the store before last time to be read.
        Slabs<BN, MODE> fill(p, first, end, step), store(p, first, end, step);
        griddep_wait();
        uint32_t ahead = 0, filled = 0;
        Slot fu, wu;
        bool ok = true;
        while (ok && store.more()) {
          for (; ahead < kBufs - 1 && fill.more(); ++ahead, ++filled) {
            if (filled >= kBufs) store_wait_read<1>();
            const uint32_t buf = staging + fu.s * kSlabBytes, bar = ready + 8 * fu.s;
            if (fill.in0 >= 0) {
              bar_expect(bar, fill.f32 || fill.in1 >= 0 ? kSlabBytes : kPlaneBytes);
              const int x = fill.col0 + fill.sl * kSlab, y = fill.row0 + my_rows;
              tma_box(buf, maps + fill.in0, bar, x, y);
              if (fill.in1 >= 0) tma_box(buf + kPlaneBytes, maps + fill.in1, bar, x, y);
            } else {
              bar_arrive(bar);
            }
            fill.next(p);
            fu.next<kBufs>();
          }
          const uint32_t buf = staging + wu.s * kSlabBytes;
          if (!bar_wait(written + 8 * wu.s, wu.parity(), limit)) {
            ok = false;
            break;
          }
          const int x = store.col0 + store.sl * kSlab, y = store.row0 + my_rows;
          if (y < store.rows && !(MODE == kSteps && empty_slab[wu.s])) {
            tma_store(maps + store.out0, buf, x, y);
            if (store.out1 >= 0) tma_store(maps + store.out1, buf + kPlaneBytes, x, y);
          }
          store_commit();
          store.next(p);
          wu.next<kBufs>();
          --ahead;
        }
        if (!ok) {
          atomicOr(p.err, kErrProductWait);
          for (; ahead > 0; --ahead, wu.next<kBufs>()) bar_wait(ready + 8 * wu.s, wu.parity(), limit);  // loads in flight
        }
        store_wait();
      }
    }
    __syncwarp();
    if (S > 1) cluster_sync();  // the epilogue warps' first one
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int ew = warp - 4;
    const int quad = warp & 3;    // the TMEM lanes this warp may read
    const int half = ew >> 2;     // warps 4-7 and 8-11 cover each quadrant once: half of every slab's columns each
    const int row = quad * 32 + lane;
    uint32_t cc = 0;
    Slot use;
    bool ok = true;
    for (int t = first, next; t < end; t = next) {
      const Place pl = place<BN, MODE>(p, t, step);
      next = pl.next;
      const Product& G = is_forward(MODE) ? p.inl[0] : *pl.P;
      const Shape sh(G, pl.k0, pl.k1, q, S);
      if (t == first) griddep_wait();
      // what the epilogue reads from HBM comes to L2 while the products run
      if constexpr (MODE != kSteps) {
        if (S == 1 && !G.swap && !p.boxes) {
          const int m = pl.row0 + my_rows + row;
          if (m < G.M) {
            const char* from = nullptr;
            int bytes = 2;
            if (is_forward(MODE) && G.add)
              from = static_cast<const char*>(G.add) + ((int64_t)m * G.ld_add + pl.col0) * 2;
            else if (MODE == kBackward && G.accumulate) {
              bytes = G.out_type == kF32 ? 4 : 2;
              from = static_cast<const char*>(G.out) + ((int64_t)m * G.ldo + pl.col0) * bytes;
            }
            if (from) {
              const int cols = G.N - pl.col0 < BN ? G.N - pl.col0 : BN;
              for (int c = half * 128; c < cols * bytes; c += 256)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(from + c));
            }
          }
        }
      }
      // in registers (no indexed access); a forward launch's only product is read as a parameter
      const Product copy = is_forward(MODE) ? Product{} : G;
      const Product& P = is_forward(MODE) ? p.inl[0] : copy;
      const uint32_t lanes = (uint32_t)(quad * 32) << 16;
      // The sums of this thread's 16 columns of the slabs in turn: from TMEM, or added up in registers chunk by chunk.
      float acc[DIRECT ? kHalf : BN / 2];
      const auto wait_sums = [&]() {
        if (ok && !bar_wait(tfull + 8 * (cc & 1u), cc >> 1 & 1u, limit)) ok = false;
        ok = __all_sync(0xffffffffu, ok);  // if not: the error word is set below, and the tile's values are not written
        fence_after();
        return ok;
      };
      const auto release_sums = [&]() {
        fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            bar_arrive_cluster(peer_addr(tempty + 8 * (cc & 1u), lead));
          else
            bar_arrive(tempty + 8 * (cc & 1u));
        }
        ++cc;
      };
      uint32_t from = 0;  // TMEM column of the slab's sums (DIRECT)
      if constexpr (DIRECT) {
        wait_sums();
        from = tmem + (cc & 1u) * BN + half * kHalf + lanes;
      } else {
#pragma unroll
        for (int k = 0; k < BN / 2; ++k) acc[k] = 0.f;
        for (int ps = 0; ps < sh.n_pass; ++ps) {
          const float scale = sh.scale(ps);
          const int chunk = sh.chunk(ps);
          for (int k0 = sh.kb0; k0 < sh.kb1; k0 += chunk) {
            if (!wait_sums()) {
              ++cc;
              continue;
            }
            const uint32_t at = tmem + (cc & 1u) * BN + half * kHalf + lanes;
            const auto add_sums = [&](auto lower) {
#pragma unroll
              for (int sl = 0; sl < kSlabs; sl += 2) {
                float v[2 * kHalf];
                tmem_ld16x2(at + sl * kSlab, at + (sl + 1) * kSlab, v);
#pragma unroll
                for (int k = 0; k < 2 * kHalf; ++k) {
                  float& a = acc[sl * kHalf + k];
                  // an infinite or NaN sum of the first planes stands: the lower ones' products with what made it so are
                  // infinite too, of either sign, or NaN
                  if (!decltype(lower)::value || fabsf(a) <= FLT_MAX) a += scale * v[k];
                }
              }
            };
            if (MODE == kBackward && ps > 0)
              add_sums(std::true_type());
            else
              add_sums(std::false_type());
            release_sums();
          }
        }
      }
      const auto load_slab = [&](int sl) {
        if constexpr (DIRECT) tmem_ld16(from + sl * kSlab, acc);
      };
      const auto next_slab = [&]() {
        if constexpr (!DIRECT) {
#pragma unroll
          for (int k = 0; k + kHalf < BN / 2; ++k) acc[k] = acc[k + kHalf];
        }
      };
      if (S > 1) {
        // one tile per cluster: the whole tile's sums go where the operands were, and are joined below
        if (ok) {
#pragma unroll 1
          for (int sl = 0; sl < kSlabs; ++sl) {
            load_slab(sl);
#pragma unroll
            for (int k = 0; k < kHalf; k += 4)
              st_shared4(ring + (row * pitch(BN) + sl * kSlab + half * kHalf + k) * 4, &acc[k]);
            next_slab();
          }
        }
        break;
      }
      bool skip = false;
      if constexpr (MODE == kSteps) {
        if (pl.parts > 1) {
          // Every part's sums go to memory, each thread's values in the thread's own place; the CTA whose part comes last
          // adds them in their order (so the result does not depend on which that is) and finishes the tile.  Nobody
          // waits for anybody.
          constexpr int kFours = BN / 8;
          float4* place4 = reinterpret_cast<float4*>(p.g_parts) + ew * 32 + lane;
          const int64_t apart = (PAIR ? 2 : 1) * kFours * (kEpiWarps * 32);
          float4* at = place4 + (pl.slot + pl.part) * apart + odd * (kFours * kEpiWarps * 32);
#pragma unroll
          for (int k = 0; k < kFours; ++k)
            __stcg(at + k * (kEpiWarps * 32), make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]));
          __threadfence();
          bar_sync_epilogue();
          if (ew == 0 && lane == 0) {  // also after a failed wait: the counters return to zero
            uint32_t* count = p.g_counts + pl.count * (PAIR ? 2 : 1) + odd;
            joins = atomicAdd(count, 1u) == (uint32_t)(pl.parts - 1);
            if (joins) *count = 0;
            __threadfence();
          }
          bar_sync_epilogue();
          skip = !joins;
          if (!skip) {
            at = place4 + pl.slot * apart + odd * (kFours * kEpiWarps * 32);
#pragma unroll
            for (int k = 0; k < kFours; ++k) {
              const float4 u = __ldcg(at + k * (kEpiWarps * 32));
              acc[4 * k] = u.x, acc[4 * k + 1] = u.y, acc[4 * k + 2] = u.z, acc[4 * k + 3] = u.w;
            }
#pragma unroll 1
            for (int part = 1; part < pl.parts; ++part) {
              at += apart;
#pragma unroll
              for (int k0 = 0; k0 < kFours; k0 += 8) {
                float4 u[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) u[k] = __ldcg(at + (k0 + k) * (kEpiWarps * 32));
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const int i = 4 * (k0 + k);
                  acc[i] += u[k].x, acc[i + 1] += u[k].y, acc[i + 2] += u[k].z, acc[i + 3] += u[k].w;
                }
              }
            }
          }
        }
      }
      bool boxes = false;
      if constexpr (BN >= 128) boxes = MODE == kSteps || p.boxes;
      if (boxes) {
        if constexpr (BN >= 128) {
          uint4 bias_ahead[2] = {};
          if constexpr (is_forward(MODE)) load_bias(P, pl.col0 + half * kHalf, bias_ahead);
#pragma unroll 1
          for (int sl = 0; sl < kSlabs && pl.col0 + sl * kSlab < P.N; ++sl, use.next<kBufs>()) {  // one copy of the code:
            // it has to stay in the instruction cache
            uint4 bias[2] = {bias_ahead[0], bias_ahead[1]};
            if (is_forward(MODE) && sl + 1 < kSlabs) load_bias(P, pl.col0 + (sl + 1) * kSlab + half * kHalf, bias_ahead);
            if (ok && !bar_wait(ready + 8 * use.s, use.parity(), limit)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            load_slab(sl);
            if (!skip)
              slab_values<MODE>(P, p, acc, bias, staging + use.s * kSlabBytes, row, half, pl.row0 + my_rows,
                                pl.col0 + sl * kSlab + half * kHalf, pl.mirror);
            fence_async();
            __syncwarp();
            if (lane == 0) {
              if (MODE == kSteps) empty_slab[use.s] = skip;
              bar_arrive(written + 8 * use.s);
            }
            next_slab();
          }
        }
      } else if constexpr (MODE != kSteps) {
#pragma unroll 1
        for (int sl = 0; sl < kSlabs; ++sl) {
          if (ok) load_slab(sl);
          bar_sync_epilogue();  // the slab before has been read
#pragma unroll
          for (int k = 0; k < kHalf; k += 4) st_shared4(staging + (row * kSlabPitch + half * kHalf + k) * 4, &acc[k]);
          next_slab();
          bar_sync_epilogue();
          const int row0 = pl.row0 + my_rows, col0 = pl.col0 + sl * kSlab;
          const OwnSums sums{staging};
          if (ok && !P.swap) write_rows<kSlab, MODE>(P, pl.P, row0, col0, lane, ew, 0, kTileM, sums);
          if (ok && P.swap) write_transposed<kSlab, MODE>(P, row0, col0, ew * 32 + lane, 0, kTileM, sums);
        }
      }
      if constexpr (DIRECT) {
        if (ok)
          release_sums();
        else
          ++cc;
      }
    }
    if (!ok && lane == 0) atomicOr(p.err, kErrProductWait);
    if (S > 1) {
      __syncwarp();
      cluster_sync();  // every CTA's sums are in its shared memory
      {  // also after a failed wait (every warp has to reach the same barriers); the values are void then
        const Place pl = place<BN, MODE>(p, first, step);
        const ClusterSums sums{ring, S, odd, PAIR ? 2 : 1};
        const Product P = *pl.P;
        if constexpr (MODE == kSteps) {
          // this CTA finishes its share of the rows; nobody else reads those sums, so its own copy can take the results
          const int share = kTileM / S;
          joined_rows<BN>(P, p, sums, pl.row0 + my_rows, pl.col0, q * share, share, ew, lane, pl.mirror);
          if (pl.mirror) {
            bar_sync_epilogue();
            joined_mirror<BN>(P, ring, pl.row0 + my_rows, pl.col0, q * share, share, ew * 32 + lane);
          }
        } else {
          // this CTA finishes its share of the rows
          const int share = kTileM / S;
          if (!P.swap)
            write_rows<BN, MODE>(P, pl.P, pl.row0 + my_rows, pl.col0, lane, ew, q * share, (q + 1) * share, sums);
          else
            write_transposed<BN, MODE>(P, pl.row0 + my_rows, pl.col0, ew * 32 + lane, q * share, share, sums);
        }
      }
    }
  }
  __syncthreads();
  if constexpr (PAIR) {
    // A pair's loads have ended when the products that read them are done; the even CTA's products arrive at the odd one's
    // barriers too, and have to before it ends.  (Nothing here is kept in registers from before: the epilogue needs them all.)
    if (threadIdx.x < kStages && !broken) {
      const uint32_t s = threadIdx.x;  // its next use would be in this lap, or in the one after
      const uint32_t lap = load_lap + (s < load_slot);
      if (!bar_wait(smem_u32(bars) + 8 * (kStages + s), (lap & 1u) ^ 1u, limit)) {
        atomicOr(p.err, kErrProductWait);
        for (int r = 0; r < 2 * p.splits; ++r) st_peer(peer_addr(smem_u32(&broken), r), 1);
      }
    }
  }
  if (PAIR || S > 1) cluster_sync();  // no CTA leaves while a peer's products or sums need it
  if constexpr (PAIR) {
    if (broken) {  // in all CTAs of the cluster: none leaves while a peer waits for its loads
      if (threadIdx.x == 0) {
        const uint32_t bar = smem_u32(bars), self = cluster_rank();
        if (drains) bar_wait(bar + 8 * (2 * kStages + 4), 0, limit);
        if (!(self & 1)) {
          Slot mine, theirs;
          mine.s = load_slot, mine.lap = load_lap;
          theirs.s = ld_peer_u32(peer_addr(smem_u32(&load_slot), self + 1));
          theirs.lap = ld_peer_u32(peer_addr(smem_u32(&load_lap), self + 1));
          end_loads<kStages>(bar, stage_bytes(BN), mine, (int)(theirs.uses<kStages>() - mine.uses<kStages>()), limit);
        }
      }
      cluster_sync();
    }
  }
  if (warp == 1) {
    fence_after();
    tmem_free<PAIR>(tmem, kCols);
  }
}

template <int BN, int MODE>
cudaError_t launch_one(const ProductLaunch& p, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> sized{0};  // devices whose copy of the kernel may use this much shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !(sized.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(product_kernel<BN, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(BN));
    if (e != cudaSuccess) return e;
    if (dev <= 63) sized.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  // a cluster per tile, or persistent CTAs or pairs
  const int cluster = (BN == 256 ? 2 : 1) * p.splits;
  const int64_t whole = (int64_t)p.n_tiles * cluster;
  const int64_t ctas = p.splits > 1 || p.g_products ? whole : std::min<int64_t>(whole, sms / cluster * cluster);
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(BN);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, product_kernel<BN, MODE>, p);
}

#ifndef DDL_PRODUCT_SELFTEST
template <int BN>
cudaError_t residency(int cluster, int* n) {
  cudaError_t e = cudaFuncSetAttribute(product_kernel<BN, kSteps>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(BN));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes(BN);
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)cluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(n, product_kernel<BN, kSteps>, &cfg);
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

#endif  // DDL_PRODUCT_SELFTEST

}  // namespace

#ifdef DDL_PRODUCT_SELFTEST
#define launch_product launch_product_selftest
#else
bool make_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t ld, int box_cols, int box_rows,
              bool bf16) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {ld * 2};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  const cuuint32_t unit[2] = {1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base),
            dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_map32(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t ld) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {ld * 4};
  const cuuint32_t box[2] = {32, (cuuint32_t)kTileM};
  const cuuint32_t unit[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, unit,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t product_residency(int sms, Residency* r) {
  r->clusters[0] = sms;
  cudaError_t e = residency<256>(2, &r->clusters[1]);
  if (e == cudaSuccess) e = residency<256>(4, &r->clusters[2]);
  if (e == cudaSuccess) e = residency<256>(8, &r->clusters[3]);
  return e;
}

#endif  // DDL_PRODUCT_SELFTEST

cudaError_t launch_product(const ProductLaunch& p, int tile_n, int sms, cudaStream_t stream) {
  if (p.n_tiles <= 0) return cudaSuccess;
  if (p.g_products) return tile_n == 256 ? launch_one<256, kSteps>(p, sms, stream) : launch_one<128, kSteps>(p, sms, stream);
  if (p.inl[0].epi == kEpiStore)
    return tile_n == 256 ? launch_one<256, kBackward>(p, sms, stream) : launch_one<128, kBackward>(p, sms, stream);
  if (p.chunked) {
    if (tile_n == 256) return launch_one<256, kForwardLong>(p, sms, stream);
    return tile_n == 128 ? launch_one<128, kForwardLong>(p, sms, stream) : launch_one<64, kForwardLong>(p, sms, stream);
  }
  if (tile_n == 256) return launch_one<256, kForward>(p, sms, stream);
  if (tile_n == 128) return launch_one<128, kForward>(p, sms, stream);
  return tile_n == 64 ? launch_one<64, kForward>(p, sms, stream) : launch_one<32, kForward>(p, sms, stream);
}

}  // namespace ddl
