// ortho_api.cu -- the C entry points of the orthogonalised update (include/ddl.h).
//
// A handle holds the matrices' places in the flat buffers, and on the device
// their planes (two X iterates in turn, the Gram matrix A, the polynomial B),
// the products of each Newton-Schulz step and the tables of their tiles.  All
// matrices go through each product in one launch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "api_util.h"
#include "ddl.h"
#include "ortho_kernels.h"
#include "product.h"

namespace {

// A launch of one kind of product over all matrices: products, tiles.
struct Stage {
  std::vector<ddl::Product> products;
  std::vector<ddl::Tile> tiles;  // the workers' first ones, then the others, linked worker by worker
  int workers = 0;
  int slots = 0, counts = 0;     // parts of tiles, tiles in parts
  ddl::Product* d_products = nullptr;
  ddl::Tile* d_tiles = nullptr;
  int tile = 128;  // rows and columns of a tile: 128, or 256 on CTA pairs
  int splits = 1;
};

enum { kGram0, kGram1, kPoly, kApply0, kApply1, kStages };  // 0/1: the X iterate read

}  // namespace

struct ddl_ortho {
  std::vector<ddl_matrix_t> mats;
  int type;
  int steps = 5;
  float coeff[3] = {3.4445f, -4.7750f, 2.0315f};
  float eps = 1e-7f;
  uint64_t extent = 0;  // elements of the flat buffers that the matrices reach
  int device = -1;
  int sms = 0;
  ddl::Residency room = {};
  bool ready = false;
  ddl::GiveUp give_up;  // of the next call's products
  uint32_t* d_err = nullptr;
  void* d_planes = nullptr;  // one block: every plane
  CUtensorMap* d_maps = nullptr;
  ddl::OrthoMatrix* d_mats = nullptr;
  ddl::OrthoItem* d_items = nullptr;
  double* d_partial = nullptr;
  float* d_parts = nullptr;      // sums of the stages' parts of tiles
  uint32_t* d_counts = nullptr;  // their counters, zero between launches
  int n_items = 0;
  Stage stage[kStages];
};

namespace {

template <typename T>
cudaError_t upload(T** dst, const T* src, size_t n) {
  cudaError_t e = ddl::device_alloc(reinterpret_cast<void**>(dst), n * sizeof(T));
  if (e == cudaSuccess) e = cudaMemcpy(*dst, src, n * sizeof(T), cudaMemcpyHostToDevice);
  return e;
}

cudaError_t release(ddl_ortho* o) {
  cudaError_t e = cudaSuccess;
  auto drop = [&e](auto** p) {
    if (*p) {
      const cudaError_t f = cudaFree(*p);  // waits for the device
      if (e == cudaSuccess) e = f;
    }
    *p = nullptr;
  };
  drop(&o->d_err);
  drop(&o->d_planes);
  drop(&o->d_maps);
  drop(&o->d_mats);
  drop(&o->d_items);
  drop(&o->d_partial);
  drop(&o->d_parts);
  drop(&o->d_counts);
  for (Stage& s : o->stage) {
    drop(&s.d_products);
    drop(&s.d_tiles);
    s = Stage();
  }
  o->ready = false;
  return e;
}

// Planes of one matrix: X twice, A, B, each hi and lo.
struct Planes {
  uint64_t x[2][2], a[2], b[2];  // element offsets in d_planes
  int64_t ldx, lds;
};

int64_t blocks_of(int64_t n, int64_t b) { return (n + b - 1) / b; }

// K blocks that the first pass of a stage's products leaves in the tensor core's truncating accumulator.  What counts
// is A A: its diagonal is one large term among small ones, and all that is added after it truncates it.  For s = 200 to
// 500 a chunk of 4 blocks there made the result's error 2 to 3.5 times a binary32 evaluation's; with these chunks it is
// 0.3 to 1.2 times that (1.5 for the longest of the smallest matrices).  One block instead of eight throughout costs
// 15 % of four 1024 x 4096, this 2 %.
int chunk_of(int stage, uint64_t s) {
  if (stage == kPoly) return s <= 640 ? 1 : 2;
  if (stage == kGram0 || stage == kGram1) return s <= 128 ? 1 : 4;
  return 8;
}

// x ~ hi + lo, so a product of two such operands is three passes; lo lo is below the last bit kept.
void split_passes(ddl::Product* P, int a_hi, int b_hi, int chunk) {
  P->n_pass = 3;
  const int a[3] = {a_hi, a_hi, a_hi + 1}, b[3] = {b_hi, b_hi + 1, b_hi};
  for (int k = 0; k < 3; ++k) {
    P->a[k] = a[k];
    P->b[k] = b[k];
    P->scale[k] = 1.f / (ddl::kPlaneScale * ddl::kPlaneScale);
  }
  P->chunk[0] = chunk;
  P->chunk[1] = 32;  // these sums are 2^-11 of the first's
}

// The tiles of every product of a stage, longest contractions first so that the last to start are short.
std::vector<ddl::Tile> tiles_of(const Stage& st, int tile, bool symmetric) {
  std::vector<ddl::Tile> tiles;
  for (int k = 0; k < (int)st.products.size(); ++k) {
    const int tm = (int)blocks_of(st.products[k].M, tile), tn = (int)blocks_of(st.products[k].N, tile);
    for (int i = 0; i < tm; ++i)
      for (int j = 0; j < (symmetric ? i + 1 : tn); ++j)
        tiles.push_back({k, i, j, symmetric && j < i, 0, (int32_t)blocks_of(st.products[k].K, ddl::kBlockK), 0, 1, 0, 0,
                         ddl::kNoTile, 0});
  }
  std::stable_sort(tiles.begin(), tiles.end(), [&st](const ddl::Tile& x, const ddl::Tile& y) {
    return st.products[x.product].K > st.products[y.product].K;
  });
  return tiles;
}

// K blocks of the busiest of `workers` CTAs (or pairs), which take the tiles in turn.
int64_t busiest(const Stage& st, const std::vector<ddl::Tile>& tiles, int workers) {
  std::vector<int64_t> load(workers, 0);
  for (size_t t = 0; t < tiles.size(); ++t) load[t % workers] += blocks_of(st.products[tiles[t].product].K, ddl::kBlockK);
  return *std::max_element(load.begin(), load.end());
}

using Lists = std::vector<std::vector<ddl::Tile>>;  // each worker's tiles

// What a tile or a part of one costs a worker, in microseconds: per K block (of all passes), and besides; a part's sums
// read back.  The blocks, a whole tile's epilogue and a launch are choose_layout's; a part and a join were chosen by the
// fit to whole runs (of (5, 2), (5, 0), (7, 0), (9, 0) and (9, 2) us for pairs the last was the fastest or within 1 %).
struct Cost {
  double block, whole, part, join;
};
constexpr int kMostParts = 8, kLeastBlocks = 4;

// Gives the workers the tiles one after the other, each up to `limit`; a tile that does not fit is cut along its
// contraction and goes on with the next worker (McNaughton's wrap-around rule).  False: they do not hold them all.
bool fill(const std::vector<ddl::Tile>& tiles, int workers, double limit, const Cost& cost, Lists* lists, int* slots,
          int* counts, int* most) {
  lists->assign(workers, {});
  *slots = *counts = *most = 0;
  int w = 0;
  double load = 0;
  for (const ddl::Tile& tile : tiles) {
    int parts = 0, in[kMostParts];
    for (int k = 0; k < tile.k1;) {
      if (w == workers) return false;
      ddl::Tile t = tile;
      t.k0 = k;
      const double need = (tile.k1 - k) * cost.block + (k ? cost.part : cost.whole);
      if (load + need <= limit) {
        load += need;
      } else {
        const int room = (int)((limit - load - cost.part) / cost.block), fit = std::min(room, tile.k1 - k - kLeastBlocks);
        if (fit < kLeastBlocks || parts == kMostParts - 1) {
          if (load == 0) return false;
          ++w;
          load = 0;
          continue;
        }
        t.k1 = k + fit;
        load = limit;
      }
      in[parts] = w;
      t.part = parts++;
      t.slot = *slots;
      t.count = *counts;
      (*lists)[w].push_back(t);
      k = t.k1;
      if (load >= limit) ++w, load = 0;
    }
    if (parts > 1) {
      for (int k = 0; k < parts; ++k) (*lists)[in[k]].back().parts = parts;
      *slots += parts;
      *counts += 1;
      *most = std::max(*most, parts);
    }
  }
  return true;
}

// Lays a stage's tiles on workers: by choose_layout, or, where the workers' shares would be uneven, cut to even ones.
// A run without and with cuts: four of 1024 x 4096 1039 and 958 us, ResNet-50's matrices 1187 and 961, one of 2304 x 2304
// 968 and 880, sets whose shares are even anyway the same.
void lay(Stage* st, bool symmetric, const ddl::Residency& room) {
  std::vector<ddl::Tile> tiles[2] = {tiles_of(*st, 128, symmetric), tiles_of(*st, 256, symmetric)};
  int64_t shortest = INT64_MAX;
  for (const ddl::Product& P : st->products) shortest = std::min(shortest, blocks_of(P.K, ddl::kBlockK));
  const ddl::Layout l = ddl::choose_layout(
      [&](int tile, int workers) { return busiest(*st, tiles[tile / 256], workers) * ddl::kMaxPasses; },
      [&](int tile) { return (int64_t)tiles[tile / 256].size(); }, shortest, room);
  st->tile = l.tile;
  st->splits = l.splits;
  Lists lists;
  double best = 0.95 * l.us;  // below 5 % cutting costs more (locality, joins) than the estimate knows
  for (int k = 0; k < 2; ++k) {
    const int workers = room.clusters[k];
    const double launch = k ? 8.8 : 4.3;
    const Cost cost = {ddl::kMaxPasses * (k ? 0.28 : 0.31), k ? 5.0 : 3.0, k ? 9.0 : 6.0, k ? 2.0 : 1.2};
    if (workers < 1 || (int64_t)tiles[k].size() > 64ll * workers) continue;  // many tiles are even enough
    double all = 0;
    for (const ddl::Tile& t : tiles[k]) all += t.k1 * cost.block + cost.whole;
    Lists trial;
    int slots, counts, most;
    double lo = all / workers, hi = best - launch;
    for (double limit = lo; hi - lo > 0.25; limit = 0.5 * (lo + hi)) {
      if (!fill(tiles[k], workers, limit, cost, &trial, &slots, &counts, &most)) {
        lo = limit;
        continue;
      }
      hi = limit;
      if (limit + launch + most * cost.join >= best) continue;
      best = limit + launch + most * cost.join;
      lists = trial;
      st->tile = k ? 256 : 128;
      st->splits = 1;
      st->slots = slots;
      st->counts = counts;
    }
  }
  if (lists.empty()) {
    const std::vector<ddl::Tile>& all = tiles[st->tile / 256];
    const int cluster = st->tile / 128 * st->splits;
    const size_t workers = st->splits > 1 ? all.size() : std::min<size_t>(all.size(), (size_t)room.clusters[cluster / 2]);
    lists.assign(workers, {});
    for (size_t t = 0; t < all.size(); ++t) lists[t % workers].push_back(all[t]);
  }
  lists.erase(std::remove_if(lists.begin(), lists.end(), [](const auto& list) { return list.empty(); }), lists.end());
  st->workers = (int)lists.size();
  for (std::vector<ddl::Tile>& list : lists) {
    // parts first: their joins then run under other tiles' products
    std::stable_partition(list.begin(), list.end(), [](const ddl::Tile& t) { return t.parts > 1; });
    st->tiles.push_back(list[0]);
  }
  for (size_t w = 0; w < lists.size(); ++w) {
    if (lists[w].size() > 1) st->tiles[w].next = (int32_t)st->tiles.size();
    for (size_t k = 1; k < lists[w].size(); ++k) {
      st->tiles.push_back(lists[w][k]);
      if (k + 1 < lists[w].size()) st->tiles.back().next = (int32_t)st->tiles.size();
    }
  }
}

// Builds the device side: planes, maps, products and tiles.
ddl_status_t build(ddl_ortho* o) {
  const int n = (int)o->mats.size();
  std::vector<Planes> pl(n);
  uint64_t at = 0;
  auto take = [&at](uint64_t elems) {
    const uint64_t here = at;
    at += (elems + 127) / 128 * 128;  // 256-byte aligned planes
    return here;
  };
  for (int i = 0; i < n; ++i) {
    const ddl_matrix_t& m = o->mats[i];
    const uint64_t s = std::min(m.rows, m.cols);
    pl[i].ldx = (int64_t)ddl::round8(m.cols);
    pl[i].lds = (int64_t)ddl::round8(s);
    for (auto& x : pl[i].x)
      for (uint64_t& v : x) v = take(m.rows * (uint64_t)pl[i].ldx);
    for (uint64_t& v : pl[i].a) v = take(s * (uint64_t)pl[i].lds);
    for (uint64_t& v : pl[i].b) v = take(s * (uint64_t)pl[i].lds);
  }
  cudaError_t e = ddl::device_alloc(&o->d_planes, at * 2);
  if (e != cudaSuccess) return ddl::status_of(e);
  uint16_t* base = static_cast<uint16_t*>(o->d_planes);

  std::vector<CUtensorMap> maps((size_t)n * 16);
  std::vector<ddl::OrthoMatrix> mats(n);
  std::vector<ddl::OrthoItem> items;
  uint64_t elems = 0;
  for (const ddl_matrix_t& m : o->mats) elems += m.rows * m.cols;
  int32_t item = ddl::kOrthoItemElems;
  while (item > ddl::kOrthoLeastElems && elems / (uint64_t)item < (uint64_t)(ddl::kOrthoItemsPerSm * o->sms)) item /= 2;
  for (int i = 0; i < n; ++i) {
    const ddl_matrix_t& m = o->mats[i];
    const uint64_t s = std::min(m.rows, m.cols);
    const Planes& p = pl[i];
    // maps 16 i + {0, 1}: X0, {2, 3}: X1, {4, 5}: A, {6, 7}: B as operands; 8 more: the same as the epilogue moves them
    const uint64_t where[8] = {p.x[0][0], p.x[0][1], p.x[1][0], p.x[1][1], p.a[0], p.a[1], p.b[0], p.b[1]};
    for (int k = 0; k < 8; ++k)
      for (int slab = 0; slab < 2; ++slab)
        if (!ddl::make_map(&maps[(size_t)i * 16 + 8 * slab + k], base + where[k], k < 4 ? m.rows : s, k < 4 ? m.cols : s,
                           (uint64_t)(k < 4 ? p.ldx : p.lds), slab ? ddl::kSlabCols : ddl::kBlockK,
                           slab ? ddl::kTileM : ddl::kBoxRows, false))
          return DDL_ERR_CUDA;
    ddl::OrthoMatrix& d = mats[i];
    d.offset = (int64_t)m.offset;
    d.ld = (int64_t)m.ld;
    const bool wide = m.rows <= m.cols;
    d.rows = (int32_t)m.rows;
    d.cols = (int32_t)m.cols;
    for (int k = 0; k < 2; ++k) {
      d.hi[k] = base + p.x[k][0];
      d.lo[k] = base + p.x[k][1];
    }
    d.ldp = p.ldx;
    d.shape_scale = wide ? 1.f : (float)std::sqrt((double)m.rows / (double)m.cols);
    d.vec = m.offset % 4 == 0 && m.ld % 4 == 0 && m.cols % 4 == 0;
    d.item0 = (int32_t)items.size();
    const int32_t cols = std::min(d.cols, item), rows = std::max(1, item / cols);
    for (int32_t r = 0; r < d.rows; r += rows)
      for (int32_t c = 0; c < d.cols; c += cols)
        items.push_back({i, r, std::min(d.rows, r + rows), c, std::min(d.cols, c + cols)});
    d.n_items = (int32_t)items.size() - d.item0;

    const int map = 16 * i;
    for (int k = 0; k < kStages; ++k) {
      ddl::Product P;
      std::memset(&P, 0, sizeof(P));
      const int xi = k == kGram1 || k == kApply1 ? 1 : 0;  // the iterate read
      if (k == kGram0 || k == kGram1) {  // A = X X^T, or X^T X when X is tall
        P.M = P.N = (int32_t)s;
        P.K = (int32_t)(wide ? m.cols : m.rows);
        P.a_mn = P.b_mn = wide ? 0 : 1;
        split_passes(&P, map + 2 * xi, map + 2 * xi, chunk_of(k, s));
        P.epi = ddl::kEpiGram;
      } else if (k == kPoly) {  // B = b A + c A A
        P.M = P.N = P.K = (int32_t)s;
        split_passes(&P, map + 4, map + 4, chunk_of(k, s));
        P.epi = ddl::kEpiPoly;
        P.c_hi = base + p.a[0];
        P.c_lo = base + p.a[1];
        P.ldc = p.lds;
      } else {  // X' = a X + B X, or a X + X B when X is tall
        P.M = (int32_t)m.rows;
        P.N = (int32_t)m.cols;
        P.K = (int32_t)s;
        P.b_mn = wide ? 1 : 0;  // X as [K][N]; B is its own transpose
        split_passes(&P, wide ? map + 6 : map + 2 * xi, wide ? map + 2 * xi : map + 6, chunk_of(k, s));
        P.epi = ddl::kEpiApply;
        P.c_hi = base + p.x[xi][0];
        P.c_lo = base + p.x[xi][1];
        P.ldc = p.ldx;
      }
      P.p_hi = base + (k == kPoly ? p.b[0] : k == kApply0 || k == kApply1 ? p.x[1 - xi][0] : p.a[0]);
      P.p_lo = base + (k == kPoly ? p.b[1] : k == kApply0 || k == kApply1 ? p.x[1 - xi][1] : p.a[1]);
      P.ldp = k == kApply0 || k == kApply1 ? p.ldx : p.lds;
      P.in0 = k == kGram0 || k == kGram1 ? -1 : k == kPoly ? map + 12 : map + 8 + 2 * xi;
      P.in1 = P.in0 < 0 ? -1 : P.in0 + 1;
      P.out0 = k == kPoly ? map + 14 : k == kApply0 || k == kApply1 ? map + 8 + 2 * (1 - xi) : map + 12;
      P.out1 = P.out0 + 1;
      P.vec = 1;  // planes always allow 4-element accesses
      o->stage[k].products.push_back(P);
    }
  }
  size_t parts = 0, counts = 0;
  for (int k = 0; k < kStages; ++k) {
    Stage& st = o->stage[k];
    lay(&st, k == kGram0 || k == kGram1 || k == kPoly, o->room);
    if (e == cudaSuccess) e = upload(&st.d_products, st.products.data(), st.products.size());
    if (e == cudaSuccess) e = upload(&st.d_tiles, st.tiles.data(), st.tiles.size());
    const size_t ctas = st.tile / 128;
    parts = std::max(parts, st.slots * ctas * ddl::kTileM * (size_t)st.tile);
    counts = std::max(counts, st.counts * ctas);
  }
  if (e == cudaSuccess && parts) e = ddl::device_alloc(reinterpret_cast<void**>(&o->d_parts), parts * sizeof(float));
  const std::vector<uint32_t> none(counts, 0);
  if (e == cudaSuccess && counts) e = upload(&o->d_counts, none.data(), counts);
  o->n_items = (int)items.size();
  if (e == cudaSuccess) e = upload(&o->d_maps, maps.data(), maps.size());
  if (e == cudaSuccess) e = upload(&o->d_mats, mats.data(), mats.size());
  if (e == cudaSuccess) e = upload(&o->d_items, items.data(), items.size());
  if (e == cudaSuccess) e = ddl::device_alloc(reinterpret_cast<void**>(&o->d_partial), items.size() * sizeof(double));
  const uint32_t zero = 0;
  if (e == cudaSuccess) e = upload(&o->d_err, &zero, 1);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);  // the caller's stream may not wait for that one
  return ddl::status_of(e);
}

// Binds the handle to the current device and builds its device side once.
ddl_status_t bind(ddl_ortho* o) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return ddl::status_of(e);
  if (o->ready) return o->device == dev ? DDL_OK : DDL_ERR_INVALID_ARG;
  e = cudaDeviceGetAttribute(&o->sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = ddl::product_residency(o->sms, &o->room);
  if (e != cudaSuccess) return ddl::status_of(e);
  ddl_status_t st;
  try {
    st = build(o);
  } catch (const std::bad_alloc&) {
    st = DDL_ERR_OOM;
  }
  if (st != DDL_OK) {
    release(o);
    return st;
  }
  o->device = dev;
  o->ready = true;
  return DDL_OK;
}

// The products of every step; the result is iterate steps & 1.
ddl_status_t products(ddl_ortho* o, cudaStream_t s) {
  ddl::ProductLaunch L = {};
  L.g_maps = o->d_maps;
  L.err = o->d_err;
  L.ca = o->coeff[0];
  L.cb = o->coeff[1];
  L.cc = o->coeff[2];
  L.give_up = o->give_up;
  o->give_up = ddl::GiveUp();  // a self-test is of one call
  for (int k = 0; k < o->steps; ++k) {
    const int order[3] = {k & 1 ? kGram1 : kGram0, kPoly, k & 1 ? kApply1 : kApply0};
    for (int kind : order) {
      const Stage& st = o->stage[kind];
      L.g_products = st.d_products;
      L.g_tiles = st.d_tiles;
      L.g_parts = o->d_parts;
      L.g_counts = o->d_counts;
      L.n_tiles = st.workers;
      L.splits = st.splits;
      L.boxes = st.splits == 1;
      const cudaError_t e = ddl::launch(L, st.tile, o->sms, s);
      if (e != cudaSuccess) return ddl::status_of(e);
    }
  }
  return DDL_OK;
}

int elem_size(int type) { return type == ddl::kF32 ? 4 : 2; }

bool aligned4(const void* p, int esize) { return reinterpret_cast<uintptr_t>(p) % (4 * (size_t)esize) == 0; }

// Preparation, products and the finishing pass.
ddl_status_t update(ddl_ortho* o, const ddl::OrthoPrep& p, ddl::OrthoFinish* f, cudaStream_t s) {
  cudaError_t e = ddl::launch_ortho_norms(p, s);
  if (e == cudaSuccess) e = ddl::launch_ortho_planes(p, s);
  if (e != cudaSuccess) return ddl::status_of(e);
  const ddl_status_t st = products(o, s);
  if (st != DDL_OK) return st;
  f->matrices = o->d_mats;
  f->items = o->d_items;
  f->n_items = o->n_items;
  f->iterate = o->steps & 1;
  return ddl::status_of(ddl::launch_ortho_finish(*f, s));
}

}  // namespace

extern "C" {

ddl_status_t ddl_ortho_create(int n_matrices, const ddl_matrix_t* matrices, ddl_dtype_t dtype, ddl_ortho_t* out) {
  if (!out) return DDL_ERR_INVALID_ARG;
  *out = nullptr;
  if (n_matrices < 1 || !matrices) return DDL_ERR_INVALID_ARG;
  if (dtype != DDL_FP32 && dtype != DDL_FP16 && dtype != DDL_BF16) return DDL_ERR_INVALID_ARG;
  constexpr uint64_t kMaxDim = 1 << 22, kMaxOffset = 1ull << 60;
  uint64_t extent = 0, tiles = 0, items = 0;
  bool unsupported = n_matrices > (1 << 20);
  for (int i = 0; i < n_matrices; ++i) {
    const ddl_matrix_t& m = matrices[i];
    if (m.rows < 1 || m.cols < 1 || m.ld < m.cols || m.offset > kMaxOffset || m.ld > kMaxOffset / m.rows)
      return DDL_ERR_INVALID_ARG;
    if (m.rows > kMaxDim || m.cols > kMaxDim) {
      unsupported = true;
      continue;
    }
    extent = std::max<uint64_t>(extent, m.offset + (m.rows - 1) * m.ld + m.cols);
    tiles += (uint64_t)blocks_of((int64_t)m.rows, 128) * (uint64_t)blocks_of((int64_t)m.cols, 128);
    items += m.rows * m.cols / (ddl::kOrthoItemElems / 2) + m.rows + 1;
  }
  if (unsupported || tiles > (1ull << 27) || items > (1ull << 27)) return DDL_ERR_UNSUPPORTED;
  ddl_ortho* o = new (std::nothrow) ddl_ortho();
  if (!o) return DDL_ERR_OOM;
  try {
    o->mats.assign(matrices, matrices + n_matrices);
    // a matrix's rows must not meet another's: compare the spans in order of their first element
    std::vector<const ddl_matrix_t*> by(n_matrices);
    for (int i = 0; i < n_matrices; ++i) by[i] = &o->mats[i];
    std::sort(by.begin(), by.end(), [](const ddl_matrix_t* a, const ddl_matrix_t* b) { return a->offset < b->offset; });
    for (int i = 0; i + 1 < n_matrices; ++i)
      if (by[i]->offset + (by[i]->rows - 1) * by[i]->ld + by[i]->cols > by[i + 1]->offset) {
        delete o;
        return DDL_ERR_INVALID_ARG;
      }
  } catch (const std::bad_alloc&) {
    delete o;
    return DDL_ERR_OOM;
  }
  o->type = dtype == DDL_FP32 ? ddl::kF32 : dtype == DDL_FP16 ? ddl::kF16 : ddl::kBF16;
  o->extent = extent;
  *out = o;
  return DDL_OK;
}

ddl_status_t ddl_ortho_set_polynomial(ddl_ortho_t o, int steps, float a, float b, float c, float eps) {
  if (!o || steps < 1 || steps > 32 || !(eps >= 0.f)) return DDL_ERR_INVALID_ARG;
  o->steps = steps;
  o->coeff[0] = a;
  o->coeff[1] = b;
  o->coeff[2] = c;
  o->eps = eps;
  return DDL_OK;
}

ddl_status_t ddl_ortho_run(ddl_ortho_t o, const void* in, void* out, void* stream) {
  if (!o || !in || !out) return DDL_ERR_INVALID_ARG;
  const int es = elem_size(o->type);
  if (reinterpret_cast<uintptr_t>(in) % es || reinterpret_cast<uintptr_t>(out) % es) return DDL_ERR_INVALID_ARG;
  const ddl::Range ri(in, o->extent * es), ro(out, o->extent * es);
  if (ri.wraps() || ro.wraps() || (in != out && ri.overlaps(ro))) return DDL_ERR_INVALID_ARG;
  ddl_status_t st = bind(o);
  if (st != DDL_OK) return st;
  if (!ddl::device_pointer(in, o->device) || !ddl::device_pointer(out, o->device)) return DDL_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  ddl::OrthoPrep p = {o->d_mats, o->d_items, o->d_partial, in,     o->type,          nullptr,
                      0.f,       0,          o->eps,       o->n_items, aligned4(in, es)};
  ddl::OrthoFinish f;
  std::memset(&f, 0, sizeof(f));
  f.out = out;
  f.type = o->type;
  f.vec = aligned4(out, es);
  return update(o, p, &f, s);
}

ddl_status_t ddl_ortho_muon(ddl_ortho_t o, const void* grad, int n_copies, float* const* param_bufs, float* mom, float lr,
                            float momentum, float weight_decay, int nesterov, void* stream) {
  if (!o || !grad || !mom || n_copies < 1 || !param_bufs) return DDL_ERR_INVALID_ARG;
  if (n_copies > ddl::kMaxCopies || o->type == ddl::kBF16) return DDL_ERR_UNSUPPORTED;
  const int es = elem_size(o->type);
  if (reinterpret_cast<uintptr_t>(grad) % es || reinterpret_cast<uintptr_t>(mom) % 4) return DDL_ERR_INVALID_ARG;
  ddl::OrthoFinish f;
  std::memset(&f, 0, sizeof(f));
  bool vec = true;
  uintptr_t at[ddl::kMaxCopies + 1];
  const uint64_t bytes = o->extent * 4;
  const ddl::Range rg(grad, o->extent * es);
  for (int r = 0; r <= n_copies; ++r) {
    float* p = r < n_copies ? param_bufs[r] : mom;
    const ddl::Range rp(p, bytes);
    if (!p || reinterpret_cast<uintptr_t>(p) % 4 || rp.wraps() || rg.wraps() || rp.overlaps(rg)) return DDL_ERR_INVALID_ARG;
    if (r < n_copies) {
      f.copies[r] = p;
      vec = vec && aligned4(p, 4);
    }
    at[r] = reinterpret_cast<uintptr_t>(p);
  }
  std::sort(at, at + n_copies + 1);
  for (int r = 0; r < n_copies; ++r)
    if (at[r] + bytes > at[r + 1]) return DDL_ERR_INVALID_ARG;
  ddl_status_t st = bind(o);
  if (st != DDL_OK) return st;
  if (!ddl::device_pointer(grad, o->device) || !ddl::device_pointer(mom, o->device)) return DDL_ERR_INVALID_ARG;
  for (int r = 0; r < n_copies; ++r)
    if (!ddl::device_pointer(param_bufs[r], o->device)) return DDL_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  ddl::OrthoPrep p = {o->d_mats, o->d_items,       o->d_partial, grad,       o->type,                              mom,
                      momentum,  nesterov ? 1 : 0, o->eps,       o->n_items, aligned4(grad, es) && aligned4(mom, 4)};
  f.lr = lr;
  f.decay = 1.f - lr * weight_decay;
  f.n_copies = n_copies;
  f.vec = vec;
  return update(o, p, &f, s);
}

ddl_status_t ddl_ortho_selftest_wait_timeout(ddl_ortho_t o, uint32_t limit_us, uint32_t products, uint32_t loads_even,
                                             uint32_t loads_odd) {
  return o && ddl::give_up_of(limit_us, products, loads_even, loads_odd, &o->give_up) ? DDL_OK : DDL_ERR_INVALID_ARG;
}

ddl_status_t ddl_ortho_check(ddl_ortho_t o, void* stream) {
  if (!o) return DDL_ERR_INVALID_ARG;
  if (!o->ready) return DDL_OK;  // no GPU call yet
  const ddl_status_t st = bind(o);
  if (st != DDL_OK) return st;
  uint32_t v = 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(&v, o->d_err, sizeof(v), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && v) e = cudaMemsetAsync(o->d_err, 0, sizeof(v), s);
  if (e == cudaSuccess && v) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return ddl::status_of(e);
  return v ? DDL_ERR_DEVICE_CHECK : DDL_OK;
}

ddl_status_t ddl_ortho_destroy(ddl_ortho_t o) {
  if (!o) return DDL_OK;
  const cudaError_t e = release(o);
  delete o;
  return ddl::status_of(e);
}

}  // extern "C"
