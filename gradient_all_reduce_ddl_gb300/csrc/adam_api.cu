// adam_api.cu -- the C entry points of the AdamW step (include/ddl.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <new>
#include <stdexcept>
#include <vector>

#include "adam_kernels.h"
#include "api_util.h"
#include "ddl.h"

struct ddl_adam {
  std::vector<ddl::AdamItem> items;
  uint64_t extent = 0;  // elements of the flat buffers that the tensors reach
  uint64_t blocks = 0;
  bool odd = false;  // a tensor does not begin at a multiple of four
  int grad_type, bits;
  double beta1 = 0.9, beta2 = 0.999, eps = 1e-8;
  int device = -1;
  int sms = 0;
  ddl::AdamItem* d_items = nullptr;
  ddl::AdamNorm* d_norm = nullptr;
  uint32_t* d_done = nullptr;
};

namespace {

cudaError_t release(ddl_adam* a) {
  cudaError_t e = cudaSuccess;
  for (void* p : {(void*)a->d_items, (void*)a->d_norm, (void*)a->d_done})
    if (p) {
      const cudaError_t f = cudaFree(p);  // waits for the device
      if (e == cudaSuccess) e = f;
    }
  a->d_items = nullptr;
  a->d_norm = nullptr;
  a->d_done = nullptr;
  return e;
}

ddl_status_t bind(ddl_adam* a) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return ddl::status_of(e);
  if (a->device >= 0) return a->device == dev ? DDL_OK : DDL_ERR_INVALID_ARG;
  const size_t bytes = a->items.size() * sizeof(ddl::AdamItem);
  e = cudaDeviceGetAttribute(&a->sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = ddl::device_alloc(reinterpret_cast<void**>(&a->d_items), bytes);
  if (e == cudaSuccess) e = ddl::device_alloc(reinterpret_cast<void**>(&a->d_norm), sizeof(ddl::AdamNorm));
  if (e == cudaSuccess) e = ddl::device_alloc(reinterpret_cast<void**>(&a->d_done), 2 * sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemcpy(a->d_items, a->items.data(), bytes, cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaMemset(a->d_done, 0, 2 * sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);  // the caller's stream may not wait for that one
  if (e != cudaSuccess) {
    release(a);
    return ddl::status_of(e);
  }
  a->device = dev;
  return DDL_OK;
}

bool aligned(const void* p, uint64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

}  // namespace

extern "C" {

ddl_status_t ddl_adam_create(int n_tensors, const ddl_tensor_t* tensors, ddl_dtype_t grad_dtype, int state_bits,
                             ddl_adam_t* out) {
  if (!out) return DDL_ERR_INVALID_ARG;
  *out = nullptr;
  if (n_tensors < 1 || !tensors || (state_bits != 32 && state_bits != 8)) return DDL_ERR_INVALID_ARG;
  if (grad_dtype != DDL_FP32 && grad_dtype != DDL_FP16 && grad_dtype != DDL_BF16) return DDL_ERR_INVALID_ARG;
  constexpr uint64_t kMost = 1ull << 48, kMostElems = 1ull << 35;  // the second: more than the states of which fill the device
  uint64_t total = 0, extent = 0, blocks = 0;
  bool odd = false;
  for (int i = 0; i < n_tensors; ++i) {
    const ddl_tensor_t& t = tensors[i];
    if (t.count < 1 || t.offset > kMost || t.count > kMost) return DDL_ERR_INVALID_ARG;
    if (!std::isfinite(t.lr_scale) || !std::isfinite(t.decay_scale)) return DDL_ERR_INVALID_ARG;
    extent = std::max(extent, (uint64_t)t.offset + t.count);
    total += t.count;
    blocks += (t.count + ddl::kAdamBlock - 1) / ddl::kAdamBlock;
    odd = odd || t.offset % 4 != 0;
    if (total > kMost) return DDL_ERR_INVALID_ARG;
  }
  if (grad_dtype == DDL_BF16 || total > kMostElems || blocks > 0xFFFFFFFFull) return DDL_ERR_UNSUPPORTED;
  ddl_adam* a = new (std::nothrow) ddl_adam();
  if (!a) return DDL_ERR_OOM;
  a->grad_type = grad_dtype == DDL_FP16 ? ddl::kF16 : ddl::kF32;
  a->bits = state_bits;
  a->extent = extent;
  a->blocks = blocks;
  a->odd = odd;
  // few elements: short items, so that every SM has some (of a GB300's: no device is asked before the first GPU call)
  constexpr uint64_t kSms = 152, kCtas = 6;
  uint64_t per = ddl::kAdamItemBlocks;
  while (per > 1 && blocks < per * kSms * kCtas) per /= 2;
  try {
    std::vector<const ddl_tensor_t*> by(n_tensors);
    for (int i = 0; i < n_tensors; ++i) by[i] = tensors + i;
    std::sort(by.begin(), by.end(), [](const ddl_tensor_t* x, const ddl_tensor_t* y) { return x->offset < y->offset; });
    for (int i = 0; i + 1 < n_tensors; ++i)
      if (by[i]->offset + by[i]->count > by[i + 1]->offset) {
        delete a;
        return DDL_ERR_INVALID_ARG;
      }
    uint64_t block = 0;
    for (int i = 0; i < n_tensors; ++i) {
      const ddl_tensor_t& t = tensors[i];
      for (uint64_t at = 0; at < t.count; at += per * ddl::kAdamBlock) {
        const uint64_t len = std::min<uint64_t>(per * ddl::kAdamBlock, t.count - at);
        a->items.push_back({t.offset + at, (uint32_t)len, (uint32_t)block, t.lr_scale, t.decay_scale});
        block += (len + ddl::kAdamBlock - 1) / ddl::kAdamBlock;
      }
    }
  } catch (const std::bad_alloc&) {
    delete a;
    return DDL_ERR_OOM;
  } catch (const std::length_error&) {
    delete a;
    return DDL_ERR_OOM;
  }
  *out = a;
  return DDL_OK;
}

ddl_status_t ddl_adam_set_betas(ddl_adam_t a, double beta1, double beta2, double eps) {
  if (!a || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !((float)eps >= FLT_MIN) || !std::isfinite((float)eps))
    return DDL_ERR_INVALID_ARG;
  a->beta1 = beta1;
  a->beta2 = beta2;
  a->eps = eps;
  return DDL_OK;
}

ddl_status_t ddl_adam_blocks(ddl_adam_t a, size_t* n) {
  if (!a || !n) return DDL_ERR_INVALID_ARG;
  *n = (size_t)a->blocks;
  return DDL_OK;
}

ddl_status_t ddl_adam_step(ddl_adam_t a, const void* grad, int n_copies, float* const* param_bufs,
                           void* const* operand_bufs, ddl_dtype_t operand_dtype, void* m, void* v, float* scales,
                           int64_t* step, float lr, float weight_decay, float grad_scale, float max_norm, float* norm,
                           void* stream) {
  if (!a || !grad || n_copies < 1 || !param_bufs || !m || !v || !step) return DDL_ERR_INVALID_ARG;
  if ((a->bits == 8) != (scales != nullptr)) return DDL_ERR_INVALID_ARG;
  if (operand_bufs && operand_dtype != DDL_FP16 && operand_dtype != DDL_BF16) return DDL_ERR_INVALID_ARG;
  if (!(max_norm >= 0.f) || !std::isfinite(max_norm)) return DDL_ERR_INVALID_ARG;
  if (n_copies > ddl::kMaxAdamCopies) return DDL_ERR_UNSUPPORTED;
  const uint64_t n = a->extent, ge = a->grad_type == ddl::kF32 ? 4 : 2, se = a->bits == 8 ? 1 : 4;
  ddl::AdamStep p = {};
  ddl::AdamCopies<ddl::kMaxAdamCopies> copies;  // the first n_copies are set
  // everything a call writes is apart from everything else
  struct Piece {
    const void* p;
    uint64_t bytes, unit;
  };
  Piece pieces[2 * ddl::kMaxAdamCopies + 6];
  int k = 0;
  pieces[k++] = {grad, n * ge, ge};
  pieces[k++] = {m, n * se, se};
  pieces[k++] = {v, n * se, se};
  pieces[k++] = {step, 8, 8};
  if (scales) pieces[k++] = {scales, a->blocks * 8, 4};
  if (norm) pieces[k++] = {norm, 4, 4};
  bool vec = aligned(grad, 4 * ge) && aligned(m, 4 * se) && aligned(v, 4 * se);
  for (int r = 0; r < n_copies; ++r) {
    if (!param_bufs[r] || (operand_bufs && !operand_bufs[r])) return DDL_ERR_INVALID_ARG;
    pieces[k++] = {copies.params[r] = param_bufs[r], n * 4, 4};
    copies.out[r] = operand_bufs ? operand_bufs[r] : nullptr;
    vec = vec && aligned(param_bufs[r], 16);
    if (operand_bufs) {
      pieces[k++] = {operand_bufs[r], n * 2, 2};
      vec = vec && aligned(operand_bufs[r], 8);
    }
  }
  for (int i = 0; i < k; ++i)
    if (!aligned(pieces[i].p, pieces[i].unit) || ddl::Range(pieces[i].p, pieces[i].bytes).wraps()) return DDL_ERR_INVALID_ARG;
  std::sort(pieces, pieces + k, [](const Piece& x, const Piece& y) { return x.p < y.p; });
  for (int i = 0; i + 1 < k; ++i)
    if (ddl::Range(pieces[i].p, pieces[i].bytes).overlaps(ddl::Range(pieces[i + 1].p, pieces[i + 1].bytes)))
      return DDL_ERR_INVALID_ARG;
  ddl_status_t st = bind(a);
  if (st != DDL_OK) return st;
  for (int i = 0; i < k; ++i)
    if (!ddl::device_pointer(pieces[i].p, a->device)) return DDL_ERR_INVALID_ARG;
  p.items = a->d_items;
  p.n_items = (int64_t)a->items.size();
  p.grad = grad;
  p.m = m;
  p.v = v;
  p.scale_m = scales;
  p.scale_v = scales ? scales + a->blocks : nullptr;
  p.step = step;
  p.norm = max_norm > 0.f || norm ? a->d_norm : nullptr;
  p.norm_out = norm;
  p.done = a->d_done;
  p.log_beta1 = std::log(a->beta1);
  p.log_beta2 = std::log(a->beta2);
  p.beta1 = (float)a->beta1;
  p.rest1 = (float)(1.0 - a->beta1);
  p.beta2 = (float)a->beta2;
  p.rest2 = (float)(1.0 - a->beta2);
  p.eps = (float)a->eps;
  p.lr = lr;
  p.weight_decay = weight_decay;
  p.grad_scale = grad_scale;
  p.max_norm = max_norm;
  p.grad_type = a->grad_type;
  p.out_type = operand_dtype == DDL_BF16 ? ddl::kBF16 : ddl::kF16;
  p.bits = a->bits;
  p.vec = vec;
  p.odd = !vec || a->odd;
  p.n_copies = n_copies;
  p.operands = operand_bufs != nullptr;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.norm && (st = ddl::status_of(ddl::launch_adam_norm(p, a->sms, s))) != DDL_OK) return st;
  return ddl::status_of(ddl::launch_adam_step(p, copies, a->sms, s));
}

ddl_status_t ddl_adam_destroy(ddl_adam_t a) {
  if (!a) return DDL_OK;
  const cudaError_t e = release(a);
  delete a;
  return ddl::status_of(e);
}

}  // extern "C"
