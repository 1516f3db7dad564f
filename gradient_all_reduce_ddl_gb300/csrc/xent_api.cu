// xent_api.cu -- the C entry points of the softmax cross entropy of a linear head (include/ddl.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "ddl.h"
#include "layer_util.h"
#include "product.h"
#include "xent.cuh"
#include "xent_kernels.h"

struct ddl_xent {
  int64_t max_tokens, n_in, vocab;
  int type;  // ddl::ElemType of x, w, bias, dx
  float smoothing;
  int device = -1;
  int sms = 0;
  ddl::Residency room = {};
  uint32_t* d_err = nullptr;
  ddl::GiveUp give_up;  // of the next call's first product
  ddl::Buffer x, w, part, part_sum, picked, planes[3], scale, resid, db, dx;
};

namespace {

using namespace ddl;

constexpr int64_t kMaxTokens = 1 << 20;
constexpr int64_t kMaxFeatures = 1 << 22;
constexpr int64_t kMaxTiles = (1ll << 31) - 1;
constexpr int64_t kFewTokens = 64;            // up to here they are the narrow side of the tiles
constexpr int64_t kMostParts = 1ll << 26;     // of a forward launch, over its tokens: 512 MB
constexpr int64_t kPieceElems = 1ll << 28;    // tokens x entries of a piece of the vocabulary: 512 MB a plane
constexpr int64_t kPieceStep = 256;           // pieces begin at whole tiles
// K blocks of logits that stay in the tensor core's truncating accumulator.  The products run on under an epilogue for two
// chunks: with short ones they wait for it.  8192 tokens, 4096 features, a vocabulary of 65,536: 2852, 2649, 2543 us with 4, 8,
// 16 blocks, and a training step of 2048 features 7634, 7281, 7119 us; relative errors of the loss 1.8, 3.7, 7.8e-7 (products in
// binary32: 6.6e-7) and of binary32 dw 1.7, 1.6, 2.0e-6 (1.75e-6).  The gradient takes the loss's chunk: what truncation takes
// from z it then takes from lse, too (with 16 blocks under a loss of 8 dw is 3.0e-6 off): 8 blocks.
// Few tokens' losses are not averaged over many: up to 64 tokens 6 blocks (16 tokens, 4096 features, 65,536 entries: 93.0, 93.3,
// 96.9, 102, 111, 136 us with 8, 6, 4, 3, 2, 1; with 6 the loss of 9 to 64 is 2.5 to 2.9e-7 off, products in binary32 3 to
// 6e-7).  Of up to 8 tokens 2 (one token over the same: of 32 losses the worst 3.8, 2.1, 1.2, 1.6e-6 off with 6, 4, 2, 1, products in
// binary32 0.9e-6; 89.3, 92.6, 106, 131 us), and 1 where the weights are few tiles (2048 features, 1000 entries: 8.5 -> 8.9 us in
// graph replay from 2).
int32_t logit_chunk(const ddl_xent* h, int64_t tokens) {
  return tokens > kFewTokens ? 8 : tokens > 8 ? 6 : blocks_of(h->vocab, kTileM) > h->sms ? 2 : 1;
}

ddl_status_t bind(ddl_xent* h) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return status_of(e);
  if (h->device >= 0) return h->device == dev ? DDL_OK : DDL_ERR_INVALID_ARG;
  uint32_t* err = nullptr;
  e = device_alloc(reinterpret_cast<void**>(&err), sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemset(err, 0, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);  // the caller's stream may not wait for that one
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = product_residency(h->sms, &h->room);
  if (e != cudaSuccess) {
    cudaFree(err);
    return status_of(e);
  }
  h->d_err = err;
  h->device = dev;
  return DDL_OK;
}

// Parts of the vocabulary that a forward launch may leave of a token: two per tile of 128 entries, or, of few tokens, up to
// eight.
int64_t most_parts(const ddl_xent* h, bool few) { return blocks_of(h->vocab, 128) * (few ? 8 : 2); }

// Tokens of a forward launch, at most.
int64_t band_of(const ddl_xent* h) { return std::max<int64_t>(256, kMostParts / most_parts(h, false) / 256 * 256); }

// Entries of a piece of the vocabulary, for a number of tokens: whole tiles, evenly shared out.
int64_t piece_of(int64_t vocab, int64_t tokens) {
  const int64_t most = std::max(kPieceStep, kPieceElems / tokens / kPieceStep * kPieceStep);
  const int64_t pieces = blocks_of(vocab, most);
  return std::min(vocab, blocks_of(blocks_of(vocab, pieces), kPieceStep) * kPieceStep);
}

// Elements of a plane: the most of any number of tokens.
size_t plane_elems(const ddl_xent* h) {
  return (size_t)std::min(h->max_tokens * (int64_t)round8((uint64_t)h->vocab), std::max(kPieceElems, h->max_tokens * kPieceStep));
}

// Sums of the bias gradient: a row per 32 tokens of a piece, or, where a contraction is split, per share of a tile's.
constexpr int64_t kSplitSums = 1 << 20;

// The checks that forward and backward share.
bool inputs_fit(const ddl_xent* h, int64_t T, const void* x, size_t ldx, const void* w, size_t ldw, const void* bias,
                const int64_t* labels) {
  return x && w && labels && fits(T, (int64_t)ldx, h->n_in) && fits(h->vocab, (int64_t)ldw, h->n_in) &&
         reinterpret_cast<uintptr_t>(x) % 2 == 0 && reinterpret_cast<uintptr_t>(w) % 2 == 0 &&
         reinterpret_cast<uintptr_t>(bias) % 2 == 0 && reinterpret_cast<uintptr_t>(labels) % 8 == 0;
}

GiveUp take_give_up(ddl_xent* h) {
  const GiveUp g = h->give_up;
  h->give_up = GiveUp();
  return g;
}

void set_softmax(const ddl_xent* h, Softmax* e, const int64_t* labels, int64_t first, const void* bias) {
  e->labels = labels;
  e->first = first;
  e->vocab = h->vocab;
  e->bias = bias ? static_cast<const uint16_t*>(bias) + first : nullptr;
  e->bias_vec = reinterpret_cast<uintptr_t>(e->bias) % 16 == 0;
}

}  // namespace

extern "C" {

ddl_status_t ddl_xent_create(size_t max_tokens, size_t in_features, size_t vocab, ddl_dtype_t dtype, float smoothing,
                             ddl_xent_t* out) {
  if (!out) return DDL_ERR_INVALID_ARG;
  *out = nullptr;
  if (max_tokens < 1 || in_features < 1 || vocab < 1 || !(smoothing >= 0.f && smoothing < 1.f)) return DDL_ERR_INVALID_ARG;
  if (dtype != DDL_FP32 && dtype != DDL_FP16 && dtype != DDL_BF16) return DDL_ERR_INVALID_ARG;
  if (dtype == DDL_FP32 || max_tokens > (size_t)kMaxTokens || in_features > (size_t)kMaxFeatures ||
      vocab > (size_t)kMaxFeatures)
    return DDL_ERR_UNSUPPORTED;
  ddl_xent* h = new (std::nothrow) ddl_xent();
  if (!h) return DDL_ERR_OOM;
  h->max_tokens = (int64_t)max_tokens;
  h->n_in = (int64_t)in_features;
  h->vocab = (int64_t)vocab;
  h->type = dtype == DDL_BF16 ? kBF16 : kF16;
  h->smoothing = smoothing;
  *out = h;
  return DDL_OK;
}

ddl_status_t ddl_xent_forward(ddl_xent_t h, size_t tokens, const void* x, size_t ldx, const void* w, size_t ldw,
                              const void* bias, const int64_t* labels, float* loss, float* lse, void* stream) {
  if (!h || tokens > (size_t)h->max_tokens) return DDL_ERR_INVALID_ARG;
  const int64_t T = (int64_t)tokens, K = h->n_in, V = h->vocab;
  if (T == 0) return DDL_OK;
  if (!inputs_fit(h, T, x, ldx, w, ldw, bias, labels) || (!loss && !lse)) return DDL_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(loss) % 4 || reinterpret_cast<uintptr_t>(lse) % 4) return DDL_ERR_INVALID_ARG;
  const Mat mx{x, T, K, (int64_t)ldx}, mw{w, V, K, (int64_t)ldw}, mb{bias, 1, V, V}, ml{labels, 1, T, T}, mo{loss, 1, T, T},
      me{lse, 1, T, T};
  const Operand outs[2] = {{mo, 4}, {me, 4}}, ins[4] = {{mx, 2}, {mw, 2}, {mb, 2}, {ml, 8}};
  if (!distinct(outs, 2, ins, 4)) return DDL_ERR_INVALID_ARG;
  ddl_status_t st = bind(h);
  if (st != DDL_OK) return st;
  for (const void* p : {x, w, bias, (const void*)labels, (const void*)loss, (const void*)lse})
    if (p && !device_pointer(p, h->device)) return DDL_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);

  const int64_t few = std::min(h->max_tokens, kFewTokens);
  const size_t parts = (size_t)std::max(most_parts(h, true) * few, most_parts(h, false) * std::min(h->max_tokens, band_of(h)));
  if ((st = need(&h->part, parts * sizeof(float2))) != DDL_OK) return st;
  if (h->smoothing > 0.f && (st = need(&h->part_sum, parts * 4)) != DDL_OK) return st;
  if ((st = need(&h->picked, (size_t)h->max_tokens * 4)) != DDL_OK) return st;
  LinearPrep prep;
  std::memset(&prep, 0, sizeof(prep));
  prep.type = h->type;
  Mat ax, aw;
  if ((st = aligned(mx, h->max_tokens, &h->x, &prep, &ax)) != DDL_OK) return st;
  if ((st = aligned(mw, V, &h->w, &prep, &aw)) != DDL_OK) return st;
  if (prep.n_packs && (st = status_of(launch_linear_prep(prep, s))) != DDL_OK) return st;

  const int64_t steps = blocks_of(K, kBlockK), band = band_of(h);
  for (int64_t t0 = 0; t0 < T; t0 += band) {
    const int64_t n = std::min(band, T - t0);
    // few tokens: their side becomes the narrow side of the tiles, and the 128-row side walks the weights
    const bool swap = n <= kFewTokens;
    int tile_n = n <= 32 ? 32 : 64, splits = 1;
    int64_t tiles = blocks_of(V, kTileM);
    int tile_rows = kTileM;
    if (swap) {
      while (splits < 8 && tiles * splits * 2 <= h->sms && steps >= 4 * splits) splits *= 2;
      // The weights are the traffic.  Where every SM has a tile or more, tiles of fewer rows may share them out more evenly:
      // the fewest rows for the busiest SM (a vocabulary of 65,536, 4096 features: 98.9 us with 128 rows, 95.2 with 120, 92.5 with
      // 112).  A block of 64 takes an SM 0.31 us however few rows it has, which is what 108 of them take from HBM: 96 rows 111 us.
      if (splits == 1 && tiles > h->sms) {
        int64_t most = blocks_of(tiles, h->sms) * tile_rows;
        for (int rows = kTileM - 8; rows >= 112; rows -= 8) {
          const int64_t busy = blocks_of(blocks_of(V, rows), h->sms) * rows;
          if (busy < most) most = busy, tile_rows = rows;
        }
        tiles = blocks_of(V, tile_rows);
      }
    } else {
      const auto count = [&](int tile) { return blocks_of(n, tile) * blocks_of(V, tile); };
      const Layout l = choose_layout([&](int tile, int workers) { return blocks_of(count(tile), workers) * steps; }, count, steps,
                                     h->room);
      tile_n = l.tile;
      splits = l.splits;
      tiles = count(tile_n);
    }
    ProductLaunch L = {};
    L.bf16 = h->type == kBF16;
    const Mat bx{static_cast<const uint16_t*>(ax.p) + t0 * ax.ld, n, K, ax.ld};
    const int narrow = std::min(tile_n, kTileM);
    if (!map_of(&L, 0, bx, kBlockK, swap ? narrow : kTileM) || !map_of(&L, 1, aw, kBlockK, swap ? tile_rows : narrow))
      return DDL_ERR_CUDA;
    Product& P = L.inl[0];
    P.M = (int32_t)(swap ? V : n);
    P.N = (int32_t)(swap ? n : V);
    P.K = (int32_t)K;
    P.n_pass = 1;
    P.a[0] = swap ? 1 : 0;
    P.b[0] = swap ? 0 : 1;
    P.scale[0] = 1.f;
    P.chunk[0] = P.chunk[1] = logit_chunk(h, T);
    P.epi = kEpiLoss;
    P.swap = swap;
    P.type = h->type;
    P.in0 = P.in1 = P.out0 = P.out1 = -1;
    L.n_inl = 1;
    L.inl_tiles[0] = L.n_tiles = (int32_t)tiles;
    L.splits = splits;
    L.tile_rows = tile_rows;
    L.err = h->d_err;
    L.give_up = take_give_up(h);
    set_softmax(h, &L.soft, labels + t0, 0, bias);
    L.soft.tokens = n;
    L.soft.part = static_cast<float2*>(h->part.p);
    L.soft.part_sum = static_cast<float*>(h->part_sum.p);
    L.soft.picked = static_cast<float*>(h->picked.p);
    if ((st = status_of(launch(L, tile_n, h->sms, s))) != DDL_OK) return st;
    XentJoin j = {};
    j.part = L.soft.part;
    j.part_sum = L.soft.part_sum;
    j.picked = L.soft.picked;
    j.ld = j.tokens = n;
    // a part per half of a tile's columns, per tile where a cluster joined its sums, or per share of a tile's entries
    j.n_parts = (int32_t)(swap ? tiles * splits : blocks_of(V, tile_n) * (splits == 1 ? 2 : 1));
    j.labels = labels + t0;
    j.vocab = V;
    j.smoothing = h->smoothing;
    j.loss = loss ? loss + t0 : nullptr;
    j.lse = lse ? lse + t0 : nullptr;
    j.err = h->d_err;
    if ((st = status_of(launch_xent_join(j, s))) != DDL_OK) return st;
  }
  return DDL_OK;
}

ddl_status_t ddl_xent_backward(ddl_xent_t h, size_t tokens, const void* x, size_t ldx, const void* w, size_t ldw,
                               const void* bias, const int64_t* labels, const float* lse, const float* dloss, void* dx,
                               size_t lddx, void* dw, size_t lddw, void* db, ddl_dtype_t grad_dtype, int accumulate,
                               void* stream) {
  if (!h || tokens > (size_t)h->max_tokens || (grad_dtype != DDL_FP32 && grad_dtype != DDL_FP16)) return DDL_ERR_INVALID_ARG;
  const int64_t T = (int64_t)tokens, K = h->n_in, V = h->vocab;
  if (!dw && !db) {
    if (T == 0) return DDL_OK;  // dx, given or not, has no elements
    if (!dx) return DDL_ERR_INVALID_ARG;
  }
  const int ge = grad_dtype == DDL_FP32 ? 4 : 2;
  if (T > 0 && (!inputs_fit(h, T, x, ldx, w, ldw, bias, labels) || !lse || (dx && !fits(T, (int64_t)lddx, K))))
    return DDL_ERR_INVALID_ARG;
  if (dw && !fits(V, (int64_t)lddw, K)) return DDL_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(dloss) % 4 || reinterpret_cast<uintptr_t>(dx) % 2 ||
      reinterpret_cast<uintptr_t>(dw) % ge || reinterpret_cast<uintptr_t>(db) % ge)
    return DDL_ERR_INVALID_ARG;
  const bool some = T > 0;
  const Mat mx{some ? x : nullptr, T, K, (int64_t)ldx}, mw{some ? w : nullptr, V, K, (int64_t)ldw},
      mb{some ? bias : nullptr, 1, V, V}, ml{some ? labels : nullptr, 1, T, T}, me{some ? lse : nullptr, 1, T, T},
      mc{some ? dloss : nullptr, 1, T, T}, mdx{dx, T, K, (int64_t)lddx}, mdw{dw, V, K, (int64_t)lddw}, mdb{db, 1, V, V};
  const Operand outs[3] = {{mdx, 2}, {mdw, ge}, {mdb, ge}},
                ins[6] = {{mx, 2}, {mw, 2}, {mb, 2}, {ml, 8}, {me, 4}, {mc, 4}};
  if (!distinct(outs, 3, ins, 6)) return DDL_ERR_INVALID_ARG;
  const int64_t piece = some ? piece_of(V, T) : V;
  if ((blocks_of(T, kTileM) + blocks_of(piece, kTileM)) * blocks_of(K, 128) * 8 > kMaxTiles) return DDL_ERR_UNSUPPORTED;
  ddl_status_t st = bind(h);
  if (st != DDL_OK) return st;
  for (const void* p : {mx.p, mw.p, mb.p, ml.p, me.p, mc.p, (const void*)dx, (const void*)dw, (const void*)db})
    if (p && !device_pointer(p, h->device)) return DDL_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!some) {  // an empty sum
    cudaError_t e = cudaSuccess;
    if (dw && !accumulate)
      e = cudaMemset2DAsync(dw, (size_t)lddw * (size_t)ge, 0, (size_t)K * (size_t)ge, (size_t)V, s);
    if (e == cudaSuccess && db && !accumulate) e = cudaMemsetAsync(db, 0, (size_t)V * (size_t)ge, s);
    return status_of(e);
  }

  // dz is kept to 16 bits of its operands' type in dx (but for the label's, see XentRound), whose own rounding is as coarse, and
  // in binary16 gradients of binary16 layers, which end 1.35 times their own rounding off (517 tokens, 771 features, 5003 entries
  // 2.8e-4; with two planes 2.1e-4 and 61.4 -> 65.6 us backward; 2048, 2048, 8192: 182 -> 228); else to two such planes, 16 or 22
  // bits, or in binary32 gradients of bfloat16 layers, if not many tokens count (planes_of), to three, 24.
  const bool f16 = h->type == kF16;
  const int dw_planes = !dw ? 0 : f16 && grad_dtype == DDL_FP16 ? 1 : !f16 && grad_dtype == DDL_FP32 ? 3 : 2;
  const int n_planes = std::max(1, dw_planes);
  for (int k = 0; k < n_planes; ++k)
    if ((st = need(&h->planes[k], plane_elems(h) * 2)) != DDL_OK) return st;
  if ((st = need(&h->scale, 3 * sizeof(float))) != DDL_OK) return st;
  const int64_t most_sums = std::max<int64_t>(kSplitSums, (int64_t)plane_elems(h) / 32 + (int64_t)round8((uint64_t)V));
  if (db && (st = need(&h->db, (size_t)most_sums * 4)) != DDL_OK) return st;
  const int64_t ld32 = (int64_t)round8((uint64_t)K);
  if (dx && ((st = need(&h->dx, (size_t)h->max_tokens * (size_t)ld32 * 4)) != DDL_OK ||
             (st = need(&h->resid, (size_t)h->max_tokens * 4)) != DDL_OK))
    return st;
  LinearPrep prep;
  std::memset(&prep, 0, sizeof(prep));
  prep.type = h->type;
  Mat ax, aw;
  if ((st = aligned(mx, h->max_tokens, &h->x, &prep, &ax)) != DDL_OK) return st;
  if ((st = aligned(mw, V, &h->w, &prep, &aw)) != DDL_OK) return st;
  if (prep.n_packs && (st = status_of(launch_linear_prep(prep, s))) != DDL_OK) return st;
  float* scale = static_cast<float*>(h->scale.p);
  const bool many = T > kScaleTokens;
  const XentScale sc = {dloss, labels, T, V, f16, n_planes, scale};
  if (many && (st = status_of(launch_xent_scale(sc, s))) != DDL_OK) return st;
  const GiveUp give_up = take_give_up(h);
  XentEnd end = {};  // what follows the products

  const int64_t ldp = (int64_t)round8((uint64_t)piece);
  for (int64_t v0 = 0; v0 < V; v0 += piece) {
    const int64_t n = std::min(piece, V - v0);
    const Mat bw{static_cast<const uint16_t*>(aw.p) + v0 * aw.ld, n, K, aw.ld};
    const Mat mp[3] = {{h->planes[0].p, T, n, ldp}, {h->planes[1].p, T, n, ldp}, {h->planes[2].p, T, n, ldp}};
    {
      const int64_t steps = blocks_of(K, kBlockK);
      const auto count = [&](int tile) { return blocks_of(T, tile) * blocks_of(n, tile); };
      const Layout l = choose_layout([&](int tile, int workers) { return blocks_of(count(tile), workers) * steps; }, count, steps,
                                     h->room);
      int splits = l.splits;
      const int64_t split_rows = blocks_of(T, kTileM) * splits, groups = splits == 1 ? blocks_of(T, 32) : split_rows;
      if (db && groups * ldp > most_sums) splits = 1;
      ProductLaunch L = {};
      L.bf16 = !f16;
      const int narrow = std::min(l.tile, kTileM);
      if (!map_of(&L, 0, ax, kBlockK, kTileM) || !map_of(&L, 1, bw, kBlockK, narrow)) return DDL_ERR_CUDA;
      for (int k = 0; k < std::min(n_planes, 2); ++k)
        if (!map_of(&L, 2 + k, mp[k], kSlabCols)) return DDL_ERR_CUDA;
      Product& P = L.inl[0];
      P.M = (int32_t)T;
      P.N = (int32_t)n;
      P.K = (int32_t)K;
      P.n_pass = 1;
      P.a[0] = 0;
      P.b[0] = 1;
      P.scale[0] = 1.f;
      P.chunk[0] = P.chunk[1] = logit_chunk(h, T);
      P.epi = kEpiGrad;
      P.type = h->type;
      P.in0 = P.in1 = -1;
      P.out0 = 2;
      P.out1 = n_planes >= 2 ? 3 : -1;
      P.p_hi = static_cast<uint16_t*>(h->planes[0].p);
      P.p_lo = static_cast<uint16_t*>(h->planes[1].p);
      P.ldp = ldp;
      L.n_inl = 1;
      L.inl_tiles[0] = L.n_tiles = (int32_t)count(l.tile);
      L.splits = splits;
      L.boxes = splits == 1;
      L.err = h->d_err;
      if (v0 == 0) L.give_up = give_up;
      set_softmax(h, &L.soft, labels, v0, bias);
      L.soft.lse = lse;
      L.soft.coef = dloss;
      L.soft.scaled = many;
      L.soft.scale = scale;
      L.soft.on = 1.f - h->smoothing;
      L.soft.off = h->smoothing / (float)V;
      L.soft.planes = n_planes;
      L.soft.third = static_cast<uint16_t*>(h->planes[2].p);
      L.soft.resid = dx ? static_cast<float*>(h->resid.p) : nullptr;
      L.soft.db = db ? static_cast<float*>(h->db.p) : nullptr;
      L.soft.ld_db = ldp;
      if ((st = status_of(launch(L, l.tile, h->sms, s))) != DDL_OK) return st;
      if (db) {
        end.bias.part = L.soft.db;
        end.bias.ld = ldp;
        end.bias.groups = splits == 1 ? blocks_of(T, 32) : blocks_of(T, kTileM) * splits;
        end.bias.cols = n;
        end.bias.scale = scale + 1;
        end.bias.db = static_cast<char*>(db) + v0 * ge;
        end.bias.f32 = ge == 4;
        end.bias.accumulate = accumulate ? 1 : 0;
      }
      // the last piece's goes with dx
      if (v0 + n < V && (st = status_of(launch_xent_end(end, s))) != DDL_OK) return st;
    }
    if (!dx && !dw) continue;

    const Mat ow{dw ? static_cast<char*>(dw) + v0 * (int64_t)lddw * ge : nullptr, n, K, (int64_t)lddw};
    const Mat ox{h->dx.p, T, ld32, ld32};  // dx's sums over the pieces, with their rows' padding
    const auto dw_count = [&](int tile) { return blocks_of(n, tile) * blocks_of(K, tile); };
    const auto dx_count = [&](int tile) { return blocks_of(T, tile) * blocks_of(K, tile); };
    // (a guess, where which tokens count decides)
    const int dw_passes = T > (int64_t)kExactTokens ? std::min(dw_planes, 2) : dw_planes;
    const int64_t dw_steps = blocks_of(T, kBlockK) * dw_passes, dx_steps = blocks_of(n, kBlockK);
    const auto layout = [&](bool with_dw, bool with_dx) {
      // the product with the longer contraction first; the workers take the tiles in turn
      const bool dw_first = with_dw && (!with_dx || dw_steps >= dx_steps);
      const auto first = [&](int tile) { return dw_first ? dw_count(tile) : dx_count(tile); };
      const auto second = [&](int tile) { return !with_dw || !with_dx ? 0 : dw_first ? dx_count(tile) : dw_count(tile); };
      const int64_t s1 = dw_first ? dw_steps : dx_steps, s2 = dw_first ? dx_steps : dw_steps;
      return choose_layout(
          [&](int tile, int workers) {
            // the first worker has the most: its tiles are 0, workers, ...
            const int64_t ones = blocks_of(first(tile), workers), all = blocks_of(first(tile) + second(tile), workers);
            return ones * s1 + (all - ones) * s2;
          },
          [&](int tile) { return first(tile) + second(tile); },
          std::min(with_dw ? blocks_of(T, kBlockK) : INT64_MAX, with_dx ? blocks_of(n, kBlockK) : INT64_MAX), h->room);
    };
    const auto add_dw = [&](ProductLaunch& L, int tile) {  // dw[v][k] = sum_t dz[t][v] x[t][k]: both operands with their rows contiguous
      Product& P = L.inl[L.n_inl];
      P.M = (int32_t)n;
      P.N = (int32_t)K;
      P.K = (int32_t)T;
      P.a_mn = P.b_mn = 1;
      P.n_pass = dw_planes;
      for (int k = 0; k < dw_planes; ++k) {
        P.a[k] = k;
        P.b[k] = 3;
        P.scale[k] = k && f16 ? 1.f / 2048.f : 1.f;
      }
      P.chunk[0] = P.chunk[1] = ge == 4 ? f32_chunk(T) : (int32_t)long_chunk(kF16);
      if (ge == 4) P.chunk[1] = 32;  // the sums of the lower plane are small
      P.epi = kEpiStore;
      P.out_type = ge == 4 ? kF32 : kF16;
      P.accumulate = accumulate ? 1 : 0;
      P.vec = ow.vec4(ge);
      P.in0 = accumulate ? 5 : -1;
      P.out0 = 5;
      P.in1 = P.out1 = -1;
      P.out = const_cast<void*>(ow.p);
      P.ldo = ow.ld;
      L.inl_tiles[L.n_inl++] = (int32_t)dw_count(tile);
    };
    const auto add_dx = [&](ProductLaunch& L, int tile) {  // dx[t][k] (+)= sum_v dz[t][v] w[v][k]
      Product& P = L.inl[L.n_inl];
      P.M = (int32_t)T;
      P.N = (int32_t)K;
      P.K = (int32_t)n;
      P.b_mn = 1;
      P.n_pass = 1;
      P.a[0] = 0;
      P.b[0] = 4;
      P.scale[0] = 1.f;
      P.chunk[0] = P.chunk[1] = (int32_t)long_chunk(h->type);
      P.epi = kEpiStore;
      P.out_type = kF32;
      P.accumulate = v0 > 0;
      P.vec = 1;
      P.in0 = v0 > 0 ? 6 : -1;
      P.out0 = 6;
      P.in1 = P.out1 = -1;
      P.out = const_cast<void*>(ox.p);
      P.ldo = ox.ld;
      L.inl_tiles[L.n_inl++] = (int32_t)dx_count(tile);
    };
    const auto products = [&](bool with_dw, bool with_dx, const Layout& l) -> ddl_status_t {
      ProductLaunch L = {};
      L.bf16 = !f16;
      L.err = h->d_err;
      L.post = scale + 1;
      if (with_dw && dw_planes == 3) L.passes = reinterpret_cast<const int32_t*>(scale + 2);
      for (int k = 0; k < n_planes; ++k)
        if (!map_of(&L, k, mp[k], kBlockK)) return DDL_ERR_CUDA;
      if ((with_dw && !map_of(&L, 3, ax, kBlockK)) || (with_dx && !map_of(&L, 4, bw, kBlockK))) return DDL_ERR_CUDA;
      const bool dw_first = with_dw && (!with_dx || dw_steps >= dx_steps);
      if (dw_first) add_dw(L, l.tile);
      if (with_dx) add_dx(L, l.tile);
      if (with_dw && !dw_first) add_dw(L, l.tile);
      L.n_tiles = L.inl_tiles[0] + L.inl_tiles[1];
      L.splits = l.splits;
      L.boxes = L.splits == 1 && (!with_dw || ((ge == 4 ? ow.tma32() : ow.tma()) && K % 8 == 0));
      if (L.boxes) {
        // a binary16 gradient's map takes the operands' element type: TMA moves its bits only
        if (with_dw && !(ge == 4 ? map32_of(&L, 5, ow) : map_of(&L, 5, ow, kSlabCols))) return DDL_ERR_CUDA;
        if (with_dx && !map32_of(&L, 6, ox)) return DDL_ERR_CUDA;
      }
      return status_of(launch(L, l.tile, h->sms, s));
    };
    // One launch for both products, or, where their contractions differ too much for that (long ones want splits), one each:
    // 517 tokens, 771 features, 5003 entries 66 and 39 us.
    const Layout both = layout(dw != nullptr, dx != nullptr);
    if (dw && dx) {
      const Layout one = layout(false, true), two = layout(true, false);
      if (one.us + two.us < both.us) {
        if ((st = products(false, true, one)) != DDL_OK || (st = products(true, false, two)) != DDL_OK) return st;
        continue;
      }
    }
    if ((st = products(dw != nullptr, dx != nullptr, both)) != DDL_OK) return st;
  }
  if (dx)
    end.round = {static_cast<const float*>(h->dx.p), ld32, static_cast<uint16_t*>(dx), (int64_t)lddx, T, K, h->type,
                 labels, V, static_cast<const float*>(h->resid.p), scale + 1, static_cast<const uint16_t*>(aw.p), aw.ld};
  return status_of(launch_xent_end(end, s));
}

ddl_status_t ddl_xent_selftest_wait_timeout(ddl_xent_t h, uint32_t limit_us, uint32_t products, uint32_t loads_even,
                                            uint32_t loads_odd) {
  return h && give_up_of(limit_us, products, loads_even, loads_odd, &h->give_up) ? DDL_OK : DDL_ERR_INVALID_ARG;
}

ddl_status_t ddl_xent_check(ddl_xent_t h, void* stream) {
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
  if (e != cudaSuccess) return status_of(e);
  return v ? DDL_ERR_DEVICE_CHECK : DDL_OK;
}

ddl_status_t ddl_xent_destroy(ddl_xent_t h) {
  if (!h) return DDL_OK;
  cudaError_t e = cudaSuccess;
  for (void* p : {(void*)h->d_err, h->x.p, h->w.p, h->part.p, h->part_sum.p, h->picked.p, h->planes[0].p, h->planes[1].p, h->planes[2].p,
                  h->scale.p, h->resid.p, h->db.p, h->dx.p})
    if (p) {
      const cudaError_t f = cudaFree(p);  // waits for the device
      if (e == cudaSuccess) e = f;
    }
  delete h;
  return status_of(e);
}

}  // extern "C"
