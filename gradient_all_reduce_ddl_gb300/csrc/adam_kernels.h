// adam_kernels.h -- launch records of the AdamW step (internal).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace ddl {

constexpr int kAdamBlock = 128;      // elements that share the scales of an 8-bit state: four per lane of a warp
constexpr int kAdamItemBlocks = 8;   // the most blocks a CTA takes at a time
constexpr int kMaxAdamCopies = 256;  // parameter copies
constexpr int kMaxNormParts = 2048;  // CTAs of the norm's pass

// Blocks of one tensor that a CTA updates at a time.
struct AdamItem {
  uint64_t begin;  // first element in the flat buffers
  uint32_t len;    // elements; only a tensor's last item ends inside a block
  uint32_t block;  // place of its first block's scales
  float lr, decay; // the tensor's factors
};

// The gradient's norm and what the step multiplies it by; on the device, made by the norm's pass.
struct AdamNorm {
  double parts[kMaxNormParts];
  float scale;
};

struct AdamStep {
  const AdamItem* items;
  int64_t n_items;
  const void* grad;
  void *m, *v;               // binary32, or e4m3 codes of m and of sqrt(v)
  float *scale_m, *scale_v;  // of every block (8-bit states)
  int64_t* step;
  AdamNorm* norm;   // NULL: no norm
  float* norm_out;  // NULL: not wanted
  uint32_t* done;   // CTAs that have ended: [0] the step's, [1] the norm's; zero between launches
  double log_beta1, log_beta2;
  float beta1, rest1, beta2, rest2;  // rest = 1 - beta
  float eps, lr, weight_decay, grad_scale, max_norm;
  int32_t grad_type;  // ElemType
  int32_t out_type;   // ElemType of the operand copies
  int32_t bits;       // of the states: 32 or 8
  int32_t vec;        // every buffer allows accesses of four elements at multiples of four
  int32_t odd;        // not so, or a tensor does not begin at one
  int32_t n_copies;
  int32_t operands;   // there are operand copies
};

// The parameter copies; launches of a few carry a shorter record (one of 4 KB takes the host longer).
template <int N>
struct AdamCopies {
  float* params[N];
  void* out[N];
};
constexpr int kFewAdamCopies = 16;

cudaError_t launch_adam_norm(const AdamStep& p, int sms, cudaStream_t stream);
cudaError_t launch_adam_step(const AdamStep& p, const AdamCopies<kMaxAdamCopies>& c, int sms, cudaStream_t stream);

}  // namespace ddl
