// xent_kernels.h -- the passes around the loss's products (internal).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace ddl {

// Joins the vocabulary's parts: lse and loss of every token.
struct XentJoin {
  const float2* part;     // [n_parts][ld]: largest logit and sum of exp(z - largest), without the label's
  const float* part_sum;  // NULL, or kSumScale times sums of the logits
  const float* picked;    // the label's logit
  int64_t ld, tokens;
  int32_t n_parts;
  const int64_t* labels;
  int64_t vocab;
  float smoothing;
  float* loss;  // NULL: not wanted
  float* lse;   // NULL: not wanted
  uint32_t* err;
};
cudaError_t launch_xent_join(const XentJoin& p, cudaStream_t stream);

// scale[0] = 1 / c, scale[1] = c, with c the largest coefficient of a token with a label (binary16: 2^-14 times that): the
// planes hold dz / c.  Where all coefficients are the same, as in a mean, dz / c of an unlikely label is nearly -1, whose
// rounding loses nothing; that of -c would be the same for every token and not average out.  And binary16 holds the dz of
// every token, small probabilities as normal numbers.
struct XentScale {
  const float* coef;  // NULL: ones
  const int64_t* labels;
  int64_t tokens, vocab;
  int32_t f16;
  int32_t planes;  // at most
  float* scale;    // [2]: as an integer, how many planes dw takes (planes_of)
};
// (Launches of up to kScaleTokens tokens make it themselves: kEpiGrad.)
constexpr int64_t kScaleTokens = 16384;
cudaError_t launch_xent_scale(const XentScale& p, cudaStream_t stream);

// db (+)= scale * the sums of `groups` rows.
struct XentBias {
  const float* part;  // [groups][ld]
  int64_t ld, groups, cols;
  const float* scale;
  void* db;
  int32_t f32, accumulate;
};

// dx: 16-bit rows of binary32 sums, to which comes what the plane's rounding took from the label's dz, times the label's row of
// w.  That one number is most of dz where the label is not likely, and its rounding would be the whole row's error.
struct XentRound {
  const float* src;
  int64_t ld;
  uint16_t* dst;
  int64_t ldd, rows, cols;
  int32_t type;
  const int64_t* labels;
  int64_t vocab;
  const float* resid;    // (x scale)
  const float* inverse;  // of the scale
  const uint16_t* w;
  int64_t ldw;
};
// Both in one launch, as far as there are any (db, rows).
struct XentEnd {
  XentBias bias;
  XentRound round;
};
cudaError_t launch_xent_end(const XentEnd& p, cudaStream_t stream);

}  // namespace ddl
