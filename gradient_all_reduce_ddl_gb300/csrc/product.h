// product.h -- launch records of the matrix products (internal).
//
// One kernel carries every product of the linear layers, of the softmax cross
// entropy and of the Newton-Schulz steps: D = sum over passes of scale * A B^T on the tensor
// cores, then an epilogue on the binary32 sums.  Passes let an operand be the
// sum of several 16-bit planes (two of binary16 hold x 2^12 = hi + lo to 22
// bits), which is how results that are kept in binary32 get products of more
// than 11 bits.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace ddl {

constexpr int kTileM = 128;      // output rows per tile
constexpr int kBlockK = 64;      // contraction elements per stage (one 128-byte swizzle row)
constexpr int kBoxRows = 64;     // rows of an operand's TMA box
constexpr int kSlabCols = 32;    // columns that the epilogue moves at a time
constexpr int kMaxPasses = 3;
// Planes of the Newton-Schulz iterates: hi = binary16(x 2^12), lo = binary16(x 2^12 - hi).  The iterates and their
// polynomials stay below 16 in magnitude (a polynomial that lets them grow past it gives NaN); the smallest lo is 2^-36.
constexpr float kPlaneScale = 4096.f;
constexpr int kMaxMaps = 8;      // tensor maps carried in the launch record
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s for each of the kernel's waits
constexpr uint32_t kNever = ~0u;

enum ElemType : int { kF32 = 0, kF16 = 1, kBF16 = 2 };
enum ActKind : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3 };
enum EpilogueKind : int {
  kEpiLinear = 0,  // z = D + bias; y = act(z) + residual
  kEpiStore = 1,   // out = D (+ out)
  kEpiGram = 2,    // planes of D, and of its transpose
  kEpiPoly = 3,    // planes of b C + c D (C, D symmetric), and of the transpose
  kEpiApply = 4,   // planes of a C + D
  kEpiLoss = 5,    // logits z = D + bias: what their softmax needs (Softmax)
  kEpiGrad = 6     // planes of the loss's gradient in the logits (Softmax)
};

// One product.  A is M x K, B is N x K; a_mn / b_mn: stored with the rows
// contiguous instead ([K][M], [K][N]).
struct Product {
  int32_t M, N, K;
  int32_t a_mn, b_mn;
  int32_t n_pass;
  int32_t a[kMaxPasses], b[kMaxPasses];  // tensor map of each pass's operands
  float scale[kMaxPasses];
  int32_t chunk[2];  // K blocks summed in the tensor core before they are added in binary32 registers: first pass, others
  int32_t epi;     // EpilogueKind
  int32_t swap;    // D is the transpose of the output: D(i, j) belongs at out[j][i]
  int32_t type;    // ElemType of bias, add, z
  int32_t act;
  int32_t out_type;
  int32_t accumulate;
  int32_t in0, in1;    // launches with box epilogues: maps of what the epilogue reads (residual, old output, C's
  int32_t out0, out1;  // planes) and writes (output, z, the result's planes); -1: none
  int32_t vec;     // every pointer and row stride of the epilogue allows 4-element accesses
  const void* bias;
  const void* add;   // residual
  int64_t ld_add;
  void* z;
  int64_t ldz;
  void* out;
  int64_t ldo;
  // Newton-Schulz: C's planes, the result's planes (row strides ldc, ldp)
  const uint16_t* c_hi;
  const uint16_t* c_lo;
  int64_t ldc;
  uint16_t* p_hi;
  uint16_t* p_lo;
  int64_t ldp;
};

// A worker's tile of a grouped launch, or a part of its contraction.
struct alignas(16) Tile {
  int32_t product, ti, tj, mirror;
  int32_t k0, k1;       // K blocks
  int32_t part, parts;  // parts > 1: the other workers' parts are added through memory
  int32_t slot, count;  // the parts' first place there, and their counter
  int32_t next;         // the worker's next tile, or kNoTile
  int32_t pad;
};
constexpr int32_t kNoTile = 0x7FFFFFFF;

// The self-test's stops, and what its waits are bounded by (else kWaitLimitNs): roles end where something would keep them
// waiting, and the others' waits run out.
struct GiveUp {
  bool armed = false;
  uint64_t wait_ns = kWaitLimitNs;
  uint32_t products = kNever;            // chunks after which a CTA's (or pair's) products stop
  uint32_t loads[2] = {kNever, kNever};  // K blocks after which a CTA's loads stop (even and odd CTA of a pair)
};

// Sums of logits are kept times this, so that those of up to 2^22 entries are numbers where their mean is one.
constexpr float kSumScale = 0x1p-24f;

// kEpiLoss and kEpiGrad: the logits are D (M tokens x N entries of the vocabulary) plus the bias.
struct Softmax {
  const int64_t* labels;
  int64_t first, vocab;   // these are the logits of entries first, first + 1, ... of a vocabulary
  const void* bias;       // NULL: none
  int32_t bias_vec;       // it begins at a 16-byte boundary
  // kEpiLoss: of every token (rows of `tokens`) and part of the vocabulary, without the label's logit
  int64_t tokens;
  float2* part;      // the largest logit and the sum of exp(z - largest)
  float* part_sum;   // NULL, or kSumScale times the sum of the logits (with the label's)
  float* picked;     // the label's logit, where it is one of these
  // kEpiGrad: dz = coef (exp(z - lse) - off - on [entry is the label]), 0 for tokens whose label is outside [0, vocab)
  const float* lse;
  const float* coef;   // NULL: ones
  int32_t scaled;      // scale[] is there (XentScale); else the launch makes it
  float* scale;        // [0] what dz's planes are multiplied by, [1] its inverse, [2] (an integer) the planes that there are
  float on, off;
  int32_t planes;      // at most, 1 to 3 (the third for bfloat16 alone)
  uint16_t* third;     // the third plane, in rows as the others'
  float* resid;        // NULL, or of every token what rounding to the first plane takes from the label's dz (x scale)
  float* db;           // NULL, or the sums of dz (x scale) over every 32 tokens, or over a split tile's shares of them
  int64_t ld_db;
};

// Launch record.  Grouped launches read products, tiles and maps from device
// memory; single launches carry up to two products and their maps here.
struct ProductLaunch {
  CUtensorMap maps[kMaxMaps];
  Product inl[2];
  int32_t n_inl;            // products in inl (0: grouped)
  int32_t inl_tiles[2];     // tiles of each
  const CUtensorMap* g_maps;
  const Product* g_products;
  const Tile* g_tiles;
  float* g_parts;           // grouped: sums of parts, 128 x tile columns a CTA
  uint32_t* g_counts;       // grouped: a counter per tile in parts and CTA; zero between launches
  int32_t n_tiles;          // grouped: workers (CTAs, pairs or clusters); worker i begins with tile i
  int32_t splits;           // CTAs of a cluster that share a tile's contraction
  int32_t boxes;            // single launches, tiles of 128 or 256 columns, splits 1: the epilogue moves boxes by TMA (in0
                            // ... out1); grouped ones with splits 1 always do
  int32_t tile_rows;        // kEpiLoss with swap, splits 1: rows of a tile, 8 to 128, a multiple of 8 (A's boxes have as many)
  int32_t chunked;          // kEpiLinear: the contraction is longer than its chunk (tiles of 64 columns or more)
  int32_t bf16;             // operands are bfloat16, else binary16
  uint32_t* err;
  const float* post;        // kEpiStore: NULL, or a further factor of the sums, in device memory
  const int32_t* passes;    // kEpiStore: NULL, or the most passes of any product, in device memory
  Softmax soft;             // kEpiLoss, kEpiGrad
  float ca, cb, cc;         // Newton-Schulz coefficients
  GiveUp give_up;           // read by launch_product_selftest's kernels only
};

// Clusters of 1, 2, 4 and 8 CTAs of the product kernel that the current device holds at a time.
struct Residency {
  int clusters[4];
};
cudaError_t product_residency(int sms, Residency* r);

// tile_n: 128, 64 or 32 output columns per 128-row tile; 256: 256 x 256 tiles on CTA pairs.  Grouped
// launches and kEpiStore take 128 or 256.
cudaError_t launch_product(const ProductLaunch& p, int tile_n, int sms, cudaStream_t stream);
// The same kernels with p.give_up's stops.
cudaError_t launch_product_selftest(const ProductLaunch& p, int tile_n, int sms, cudaStream_t stream);

// Tensor map of a row-major 16-bit matrix (rows x cols, ld elements between rows; 16-byte aligned base and row stride):
// boxes of 64 columns (operands, 128-byte swizzle) or 32 (the epilogue's slabs, 64-byte swizzle) x box_rows.
bool make_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t ld, int box_cols, int box_rows,
              bool bf16);

// The same of a binary32 matrix, boxes of 32 columns x 128 rows (kEpiStore's output).
bool make_map32(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t ld);

// Error word bits of these kernels.
enum : uint32_t { kErrProductWait = 16u, kErrLabel = 32u };

}  // namespace ddl
