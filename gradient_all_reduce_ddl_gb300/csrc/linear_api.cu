// linear_api.cu -- the C entry points of the linear layers (include/ddl.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>

#include "ddl.h"
#include "layer_util.h"
#include "linear_kernels.h"
#include "product.h"

struct ddl_linear {
  int64_t max_tokens, n_in, n_out;
  int type;  // ddl::ElemType of x, w, y
  int act;
  int device = -1;
  int sms = 0;
  ddl::Residency room = {};
  uint32_t* d_err = nullptr;
  ddl::GiveUp give_up;  // of the next launch
  ddl::Buffer x, w, dz[ddl::kMaxPlanes], partial, done;
};

namespace {

using namespace ddl;

constexpr int64_t kMaxFeatures = 1 << 22;
// Longest sums over tokens: a tile's takes 2^20 blocks x 3 planes x 0.35 us, about half of what a kernel's waits allow.
constexpr int64_t kMaxTokens = 1 << 26;
// What a tensor map and a tile index can address.
constexpr int64_t kMaxTiles = (1ll << 31) - 1;

ddl_status_t bind(ddl_linear* h) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return ddl::status_of(e);
  if (h->device >= 0) return h->device == dev ? DDL_OK : DDL_ERR_INVALID_ARG;
  uint32_t* err = nullptr;
  e = ddl::device_alloc(reinterpret_cast<void**>(&err), sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemset(err, 0, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);  // the caller's stream may not wait for that one
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = ddl::product_residency(h->sms, &h->room);
  if (e != cudaSuccess) {
    cudaFree(err);
    return ddl::status_of(e);
  }
  h->d_err = err;
  h->device = dev;
  return DDL_OK;
}

// A self-test is of one launch.
ddl::GiveUp take_give_up(ddl_linear* h) {
  const ddl::GiveUp g = h->give_up;
  h->give_up = ddl::GiveUp();
  return g;
}

}  // namespace

extern "C" {

ddl_status_t ddl_linear_create(size_t max_tokens, size_t in_features, size_t out_features, ddl_dtype_t dtype,
                               ddl_act_t act, ddl_linear_t* out) {
  if (!out) return DDL_ERR_INVALID_ARG;
  *out = nullptr;
  if (max_tokens < 1 || in_features < 1 || out_features < 1) return DDL_ERR_INVALID_ARG;
  if (act < DDL_ACT_NONE || act > DDL_ACT_SILU) return DDL_ERR_INVALID_ARG;
  if (dtype != DDL_FP32 && dtype != DDL_FP16 && dtype != DDL_BF16) return DDL_ERR_INVALID_ARG;
  if (dtype == DDL_FP32 || max_tokens > (size_t)kMaxTokens || in_features > (size_t)kMaxFeatures ||
      out_features > (size_t)kMaxFeatures)
    return DDL_ERR_UNSUPPORTED;
  ddl_linear* h = new (std::nothrow) ddl_linear();
  if (!h) return DDL_ERR_OOM;
  h->max_tokens = (int64_t)max_tokens;
  h->n_in = (int64_t)in_features;
  h->n_out = (int64_t)out_features;
  h->type = dtype == DDL_BF16 ? ddl::kBF16 : ddl::kF16;
  h->act = (int)act;
  *out = h;
  return DDL_OK;
}

ddl_status_t ddl_linear_forward(ddl_linear_t h, size_t tokens, const void* x, size_t ldx, const void* w, size_t ldw,
                                const void* bias, const void* residual, size_t ldr, void* z, size_t ldz, void* y,
                                size_t ldy, void* stream) {
  if (!h || tokens > (size_t)h->max_tokens) return DDL_ERR_INVALID_ARG;
  const int64_t T = (int64_t)tokens, K = h->n_in, N = h->n_out;
  if (T == 0) return DDL_OK;
  if (!x || !w || !y) return DDL_ERR_INVALID_ARG;
  if (!fits(T, (int64_t)ldx, K) || !fits(N, (int64_t)ldw, K) || !fits(T, (int64_t)ldy, N) ||
      (residual && !fits(T, (int64_t)ldr, N)) || (z && !fits(T, (int64_t)ldz, N)))
    return DDL_ERR_INVALID_ARG;
  const Mat mx{x, T, K, (int64_t)ldx}, mw{w, N, K, (int64_t)ldw}, my{y, T, N, (int64_t)ldy},
      mz{z, T, N, (int64_t)ldz}, mr{residual, T, N, (int64_t)ldr}, mb{bias, 1, N, N};
  for (const Mat* m : {&mx, &mw, &my, &mz, &mr, &mb})
    if (reinterpret_cast<uintptr_t>(m->p) % 2) return DDL_ERR_INVALID_ARG;
  // y may be the residual itself (each element is read before it is written, by the same thread)
  const bool in_place = residual && residual == y && (ldr == ldy || T == 1);  // one row: its stride says nothing
  const Operand outs[2] = {{my, 2}, {mz, 2}}, ins[4] = {{mx, 2}, {mw, 2}, {mb, 2}, {in_place ? Mat{nullptr, 0, 0, 1} : mr, 2}};
  if (!distinct(outs, 2, ins, 4)) return DDL_ERR_INVALID_ARG;

  // Few tokens: their side becomes the narrow side of the tiles, 32 or 64 wide, and the 128-row side
  // walks the weights, which are the traffic then.
  int tile_n = T <= 32 ? 32 : T <= 64 ? 64 : 128;
  const bool swap = tile_n < 128;
  int64_t tiles = swap ? blocks_of(N, ddl::kTileM) : blocks_of(T, ddl::kTileM) * blocks_of(N, tile_n);
  if (tiles * 8 > kMaxTiles) return DDL_ERR_UNSUPPORTED;

  ddl_status_t st = bind(h);
  if (st != DDL_OK) return st;
  const int64_t steps = blocks_of(K, ddl::kBlockK);
  int splits = 1;
  if (swap) {
    // the weights come from HBM at the SMs' joint rate: as many CTAs as there are SMs, two blocks each at least
    while (splits < 8 && tiles * splits * 2 <= h->sms && steps >= 4 * splits) splits *= 2;
  } else {
    const auto count = [&](int tile) { return blocks_of(T, tile) * blocks_of(N, tile); };
    const ddl::Layout l = ddl::choose_layout(
        [&](int tile, int workers) { return blocks_of(count(tile), workers) * steps; }, count, steps, h->room);
    tile_n = l.tile;
    splits = l.splits;
    tiles = count(tile_n);
  }
  // a contraction beyond what may stay in the accumulator has a kernel of its own, whose narrowest tile is 64 wide (binary16
  // with and without chunks: 16 tokens, 524,288 -> 1024 283 and 282 us; 2048, 32,768 -> 4096 with GELU, residual and z 363
  // and 353)
  const int64_t chunk = long_chunk(h->type);
  const bool chunked = blocks_of(steps, splits) > chunk;
  if (chunked) tile_n = std::max(tile_n, 64);
  for (const void* p : {x, w, bias, residual, (const void*)z, (const void*)y})
    if (p && !ddl::device_pointer(p, h->device)) return DDL_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  Mat ax, aw;
  ddl::LinearPrep prep;
  std::memset(&prep, 0, sizeof(prep));
  prep.type = h->type;
  if ((st = aligned(mx, h->max_tokens, &h->x, &prep, &ax)) != DDL_OK) return st;
  if ((st = aligned(mw, N, &h->w, &prep, &aw)) != DDL_OK) return st;
  if (prep.n_packs && (st = ddl::status_of(ddl::launch_linear_prep(prep, s))) != DDL_OK) return st;

  ddl::ProductLaunch L = {};
  L.bf16 = h->type == ddl::kBF16;
  // boxes of a tile's rows
  const int narrow = std::min(tile_n, ddl::kTileM);
  if (!map_of(&L, 0, ax, ddl::kBlockK, swap ? narrow : ddl::kTileM) || !map_of(&L, 1, aw, ddl::kBlockK, swap ? ddl::kTileM : narrow))
    return DDL_ERR_CUDA;
  ddl::Product& P = L.inl[0];
  P.M = (int32_t)(swap ? N : T);
  P.N = (int32_t)(swap ? T : N);
  P.K = (int32_t)K;
  P.n_pass = 1;
  P.a[0] = swap ? 1 : 0;
  P.b[0] = swap ? 0 : 1;
  P.scale[0] = 1.f;
  P.chunk[0] = P.chunk[1] = (int32_t)(chunked ? chunk : steps);
  P.epi = ddl::kEpiLinear;
  P.swap = swap;
  P.type = h->type;
  P.act = h->act;
  P.vec = my.vec4(2) && (!z || mz.vec4(2)) && (!residual || mr.vec4(2)) && reinterpret_cast<uintptr_t>(bias) % 8 == 0;
  P.bias = bias;
  P.add = residual;
  P.ld_add = mr.ld;
  P.z = z;
  P.ldz = mz.ld;
  P.out = y;
  P.ldo = my.ld;
  L.n_inl = 1;
  L.inl_tiles[0] = (int32_t)tiles;
  L.n_tiles = (int32_t)tiles;
  L.splits = splits;
  L.chunked = chunked;
  L.err = h->d_err;
  L.give_up = take_give_up(h);
  P.in0 = P.in1 = P.out0 = P.out1 = -1;
  // rows that TMA can address, of whole 16-byte pieces, let the epilogue move whole boxes
  L.boxes = !swap && L.splits == 1 && N % 8 == 0 && my.tma() && (!z || mz.tma()) && (!residual || mr.tma()) &&
            reinterpret_cast<uintptr_t>(bias) % 16 == 0;
  if (L.boxes) {
    P.out0 = 2;
    if (!map_of(&L, 2, my, ddl::kSlabCols)) return DDL_ERR_CUDA;
    if (z) P.out1 = 3;
    if (z && !map_of(&L, 3, mz, ddl::kSlabCols)) return DDL_ERR_CUDA;
    if (residual) P.in0 = 4;
    if (residual && !map_of(&L, 4, mr, ddl::kSlabCols)) return DDL_ERR_CUDA;
  }
  return ddl::status_of(ddl::launch(L, tile_n, h->sms, s));
}

ddl_status_t ddl_linear_backward(ddl_linear_t h, size_t tokens, const void* dy, size_t ldy, const void* x, size_t ldx,
                                 const void* w, size_t ldw, const void* z, size_t ldz, void* dx, size_t lddx, void* dw,
                                 size_t lddw, void* db, ddl_dtype_t grad_dtype, int accumulate, void* stream) {
  if (!h || tokens > (size_t)h->max_tokens || (grad_dtype != DDL_FP32 && grad_dtype != DDL_FP16)) return DDL_ERR_INVALID_ARG;
  const int64_t T = (int64_t)tokens, K = h->n_in, N = h->n_out;
  if (!dw && !db) {
    if (T == 0) return DDL_OK;  // dx, given or not, has no elements
    if (!dx) return DDL_ERR_INVALID_ARG;
  }
  const int ge = grad_dtype == DDL_FP32 ? 4 : 2;
  if (T > 0 && (!dy || (dw && !x) || (dx && !w) || (h->act != ddl::kActNone && !z))) return DDL_ERR_INVALID_ARG;
  const bool has_z = h->act != ddl::kActNone;
  if (!fits(N, (int64_t)lddw, K) && dw) return DDL_ERR_INVALID_ARG;
  if (T > 0 && (!fits(T, (int64_t)ldy, N) || (dw && !fits(T, (int64_t)ldx, K)) || (dx && !fits(N, (int64_t)ldw, K)) ||
                (has_z && !fits(T, (int64_t)ldz, N)) || (dx && !fits(T, (int64_t)lddx, K))))
    return DDL_ERR_INVALID_ARG;
  const Mat mdy{dy, T, N, (int64_t)ldy}, mx{dw ? x : nullptr, T, K, (int64_t)ldx}, mw{dx ? w : nullptr, N, K, (int64_t)ldw},
      mz{has_z ? z : nullptr, T, N, (int64_t)ldz}, mdx{dx, T, K, (int64_t)lddx}, mdw{dw, N, K, (int64_t)lddw},
      mdb{db, 1, N, N};
  for (const Mat* m : {&mdy, &mx, &mw, &mz, &mdx})
    if (reinterpret_cast<uintptr_t>(m->p) % 2) return DDL_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(dw) % ge || reinterpret_cast<uintptr_t>(db) % ge) return DDL_ERR_INVALID_ARG;
  const Operand outs[3] = {{mdx, 2}, {mdw, ge}, {mdb, ge}}, ins[4] = {{mdy, 2}, {mx, 2}, {mw, 2}, {mz, 2}};
  if (!distinct(outs, 3, ins, 4)) return DDL_ERR_INVALID_ARG;

  int64_t dx_tiles = dx ? blocks_of(T, ddl::kTileM) * blocks_of(K, 128) : 0;
  int64_t dw_tiles = dw ? blocks_of(N, ddl::kTileM) * blocks_of(K, 128) : 0;
  if ((dx_tiles + dw_tiles) * 8 > kMaxTiles) return DDL_ERR_UNSUPPORTED;
  ddl_status_t st = bind(h);
  if (st != DDL_OK) return st;
  for (const void* p : {mdy.p, mx.p, mw.p, mz.p, (const void*)dx, (const void*)dw, (const void*)db})
    if (p && !ddl::device_pointer(p, h->device)) return DDL_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // an empty sum
    cudaError_t e = cudaSuccess;
    if (dw && !accumulate)
      e = cudaMemset2DAsync(dw, (size_t)lddw * (size_t)ge, 0, (size_t)K * (size_t)ge, (size_t)N, s);
    if (e == cudaSuccess && db && !accumulate) e = cudaMemsetAsync(db, 0, (size_t)N * (size_t)ge, s);
    return ddl::status_of(e);
  }

  // dz: dy itself where it can be; else planes of dy act'(z).  GELU's and SiLU's slopes are not 16-bit numbers, and
  // neither are their products with dy: a binary32 gradient sums 22 (binary16) or 24 (bfloat16) bits of dz, a 16-bit
  // result 22 or 16, so that its own rounding is all it loses.  One plane for 16-bit results would save a product each
  // (8192 tokens, 2048 -> 8192, bfloat16: 909 us become 776; 4096 -> 4096, binary16 throughout: 770 become 404) at 1.4
  // times their error, and in binary16 small gradients would fall below its normal range (dw 2.5 % off for dy ~ 1e-6)
  // and large ones overflow.  The number does not depend on the tokens: neither does a layer's precision, nor its workspace.
  const bool curved = h->act == ddl::kActGelu || h->act == ddl::kActSilu;
  const bool f16 = h->type == ddl::kF16;
  const int dw_planes = !dw ? 0 : !curved ? 1 : grad_dtype == DDL_FP32 && !f16 ? 3 : 2;
  const int dx_planes = !dx ? 0 : curved ? 2 : 1;
  const bool own_dz = (dx || dw) && (has_z || !mdy.tma());
  const int n_planes = own_dz ? std::max(dw_planes, dx_planes) : 0;
  const int64_t ldp = own_dz ? (int64_t)ddl::round8((uint64_t)N) : mdy.ld;
  for (int k = 0; k < n_planes; ++k)
    if ((st = need(&h->dz[k], (size_t)h->max_tokens * (size_t)ldp * 2)) != DDL_OK) return st;
  ddl::LinearPrep prep;
  std::memset(&prep, 0, sizeof(prep));
  prep.type = h->type;
  Mat ax, aw;
  if (dw && (st = aligned(mx, h->max_tokens, &h->x, &prep, &ax)) != DDL_OK) return st;
  if (dx && (st = aligned(mw, N, &h->w, &prep, &aw)) != DDL_OK) return st;
  if (n_planes || db) {
    prep.has_dz = 1;
    prep.dy = dy;
    prep.ldy = mdy.ld;
    prep.z = mz.p;
    prep.ldz = mz.ld;
    prep.rows = T;
    prep.cols = N;
    prep.block_rows = (int32_t)ddl::dz_rows(T);
    prep.act = h->act;
    prep.n_planes = n_planes;
    for (int k = 0; k < n_planes; ++k) prep.planes[k] = static_cast<uint16_t*>(h->dz[k].p);
    prep.ldp = ldp;
    prep.vec = mdy.tma() && (!has_z || mz.tma()) && N % 8 == 0;
  }
  if (db) {
    const size_t done = (size_t)blocks_of(N, ddl::kDzCols) * 4;
    if ((st = need(&h->partial, (size_t)ddl::dz_row_blocks(h->max_tokens) * (size_t)N * 4)) != DDL_OK) return st;
    if (!h->done.p) {
      if ((st = need(&h->done, done)) != DDL_OK) return st;
      if ((st = ddl::status_of(cudaMemsetAsync(h->done.p, 0, done, s))) != DDL_OK) {
        cudaFree(h->done.p);
        h->done.p = nullptr;
        h->done.bytes = 0;
        return st;
      }
    }
    prep.db = db;
    prep.db_f32 = grad_dtype == DDL_FP32;
    prep.accumulate = accumulate ? 1 : 0;
    prep.partial = static_cast<float*>(h->partial.p);
    prep.done = static_cast<uint32_t*>(h->done.p);
  }
  if ((st = ddl::status_of(ddl::launch_linear_prep(prep, s))) != DDL_OK) return st;
  if (!dx && !dw) return DDL_OK;

  ddl::ProductLaunch L = {};
  L.bf16 = !f16;
  L.err = h->d_err;
  L.give_up = take_give_up(h);
  const int maps = std::max(1, n_planes);
  for (int k = 0; k < maps; ++k)
    if (!map_of(&L, k, n_planes ? Mat{h->dz[k].p, T, N, ldp} : mdy, ddl::kBlockK)) return DDL_ERR_CUDA;
  if ((dw && !map_of(&L, 3, ax, ddl::kBlockK)) || (dx && !map_of(&L, 4, aw, ddl::kBlockK))) return DDL_ERR_CUDA;
  // the product with the longer contraction first; the workers take the tiles in turn
  const auto dw_count = [&](int tile) { return dw ? blocks_of(N, tile) * blocks_of(K, tile) : 0; };
  const auto dx_count = [&](int tile) { return dx ? blocks_of(T, tile) * blocks_of(K, tile) : 0; };
  const int64_t dw_steps = blocks_of(T, ddl::kBlockK) * dw_planes, dx_steps = blocks_of(N, ddl::kBlockK) * dx_planes;
  const bool dw_first = dw && (!dx || dw_steps >= dx_steps);
  const ddl::Layout l = ddl::choose_layout(
      [&](int tile, int workers) {
        const int64_t one = dw_first ? dw_count(tile) : dx_count(tile), two = dw_first ? dx_count(tile) : dw_count(tile);
        const int64_t s1 = dw_first ? dw_steps : dx_steps, s2 = dw_first ? dx_steps : dw_steps;
        int64_t most = 0;
        for (int64_t i = 0; i < workers; ++i) {  // worker i's tiles are i, i + workers, ...
          const int64_t mine = one + two > i ? (one + two - i - 1) / workers + 1 : 0, first = one > i ? (one - i - 1) / workers + 1 : 0;
          most = std::max(most, first * s1 + (mine - first) * s2);
        }
        return most;
      },
      [&](int tile) { return dw_count(tile) + dx_count(tile); },
      std::min(dw ? blocks_of(T, ddl::kBlockK) : INT64_MAX, dx ? blocks_of(N, ddl::kBlockK) : INT64_MAX), h->room);
  const int tile_n = l.tile;
  dw_tiles = dw_count(tile_n);
  dx_tiles = dx_count(tile_n);
  const auto add_dw = [&]() {  // dw[n][k] = sum_t dz[t][n] x[t][k]: both operands with their rows contiguous
    ddl::Product& P = L.inl[L.n_inl];
    P.M = (int32_t)N;
    P.N = (int32_t)K;
    P.K = (int32_t)T;
    P.a_mn = P.b_mn = 1;
    P.n_pass = dw_planes;
    for (int k = 0; k < dw_planes; ++k) {
      P.a[k] = k;
      P.b[k] = 3;
      P.scale[k] = ddl::plane_scale(h->type, maps, k);
    }
    P.chunk[0] = P.chunk[1] = grad_dtype == DDL_FP32 ? f32_chunk(T) : (int32_t)long_chunk(ddl::kF16);
    if (grad_dtype == DDL_FP32) P.chunk[1] = 32;  // the sums of lower planes are small
    P.epi = ddl::kEpiStore;
    P.out_type = grad_dtype == DDL_FP32 ? ddl::kF32 : ddl::kF16;
    P.accumulate = accumulate ? 1 : 0;
    P.vec = mdw.vec4(ge);
    P.in0 = accumulate ? 5 : -1;
    P.out0 = 5;
    P.in1 = P.out1 = -1;
    P.out = dw;
    P.ldo = mdw.ld;
    L.inl_tiles[L.n_inl++] = (int32_t)dw_tiles;
  };
  const auto add_dx = [&]() {  // dx[t][k] = sum_n dz[t][n] w[n][k]
    ddl::Product& P = L.inl[L.n_inl];
    P.M = (int32_t)T;
    P.N = (int32_t)K;
    P.K = (int32_t)N;
    P.b_mn = 1;
    P.n_pass = dx_planes;
    for (int k = 0; k < dx_planes; ++k) {
      P.a[k] = k;
      P.b[k] = 4;
      P.scale[k] = ddl::plane_scale(h->type, maps, k);
    }
    P.chunk[0] = P.chunk[1] = (int32_t)long_chunk(h->type);
    P.epi = ddl::kEpiStore;
    P.out_type = h->type;
    P.vec = mdx.vec4(2);
    P.out0 = 6;
    P.in0 = P.in1 = P.out1 = -1;
    P.out = dx;
    P.ldo = mdx.ld;
    L.inl_tiles[L.n_inl++] = (int32_t)dx_tiles;
  };
  if (dw && dw_first) add_dw();
  if (dx) add_dx();
  if (dw && !dw_first) add_dw();
  L.n_tiles = L.inl_tiles[0] + L.inl_tiles[1];
  L.splits = l.splits;
  L.boxes = L.splits == 1 && (!dw || (ge == 4 ? mdw.tma32() : mdw.tma())) && (!dx || mdx.tma()) &&
            K % 8 == 0;
  if (L.boxes) {
    // a binary16 gradient's map takes the operands' element type: TMA moves its bits only
    if (dw && !(ge == 4 ? map32_of(&L, 5, mdw) : map_of(&L, 5, mdw, ddl::kSlabCols))) return DDL_ERR_CUDA;
    if (dx && !map_of(&L, 6, mdx, ddl::kSlabCols)) return DDL_ERR_CUDA;
  }
  return ddl::status_of(ddl::launch(L, tile_n, h->sms, s));
}

ddl_status_t ddl_linear_selftest_wait_timeout(ddl_linear_t h, uint32_t limit_us, uint32_t products, uint32_t loads_even,
                                              uint32_t loads_odd) {
  return h && ddl::give_up_of(limit_us, products, loads_even, loads_odd, &h->give_up) ? DDL_OK : DDL_ERR_INVALID_ARG;
}

ddl_status_t ddl_linear_check(ddl_linear_t h, void* stream) {
  if (!h) return DDL_ERR_INVALID_ARG;
  if (h->device < 0) return DDL_OK;  // no GPU call yet
  ddl_status_t st = bind(h);
  if (st != DDL_OK) return st;
  uint32_t v = 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(&v, h->d_err, sizeof(v), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && v) e = cudaMemsetAsync(h->d_err, 0, sizeof(v), s);
  if (e == cudaSuccess && v) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return ddl::status_of(e);
  return v ? DDL_ERR_DEVICE_CHECK : DDL_OK;
}

ddl_status_t ddl_linear_destroy(ddl_linear_t h) {
  if (!h) return DDL_OK;
  cudaError_t e = cudaSuccess;
  for (void* p : {(void*)h->d_err, h->x.p, h->w.p, h->dz[0].p, h->dz[1].p, h->dz[2].p, h->partial.p, h->done.p})
    if (p) {
      const cudaError_t f = cudaFree(p);  // waits for the device
      if (e == cudaSuccess) e = f;
    }
  delete h;
  return ddl::status_of(e);
}

}  // extern "C"
