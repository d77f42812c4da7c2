// C ABI of the operators around the expert block in a learner's step: argument checks
// before anything is enqueued.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "nvfp4moe.h"
#include "launch.h"

using namespace nvfp4;

namespace {

constexpr int64_t kMaxVocab = 1 << 20;
constexpr int kMaxList = 128;
constexpr int64_t kMaxRows = (int64_t)1 << 24;   // eight CTAs a row, 64 backward tiles: below 2^31 in all

bool dtype_ok(nvfp4_act_dtype d) { return d == NVFP4_ACT_BF16 || d == NVFP4_ACT_F32 || d == NVFP4_ACT_F16; }
int elt_bytes(nvfp4_act_dtype d) { return d == NVFP4_ACT_F32 ? 4 : 2; }
bool aligned(const void* p, int bytes) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool aligned_or_null(const void* p, int bytes) { return p == nullptr || aligned(p, bytes); }
nvfp4_status from_cuda(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

// What every call over rows of logits asks of them.
nvfp4_status logits_check(nvfp4_act_dtype dtype, int64_t T, int64_t V, int64_t ld, float scale) {
  if (!dtype_ok(dtype) || T < 0 || V <= 0 || ld < V) return NVFP4_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return NVFP4_ERR_INVALID_ARG;
  if (V > kMaxVocab || T > kMaxRows) return NVFP4_ERR_UNSUPPORTED;
  return NVFP4_OK;
}

// [T, ld] and [T, ldo] of `e`-byte elements: the same memory row by row, or no byte in common.
bool same_or_disjoint(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t T, int64_t cols, int e) {
  if (a == b) return lda == ldb;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const uintptr_t a1 = a0 + static_cast<uintptr_t>(((T - 1) * lda + cols) * e);
  const uintptr_t b1 = b0 + static_cast<uintptr_t>(((T - 1) * ldb + cols) * e);
  return a1 <= b0 || b1 <= a0;
}

}  // namespace

extern "C" {

nvfp4_status token_logprobs(const void* logits, nvfp4_act_dtype dtype, int64_t T, int64_t V, int64_t ld,
                            const int32_t* targets, int32_t ignore_index, float scale, int32_t top_k, float* logprob,
                            float* lse, float* entropy, float* top_logprob, int32_t* top_ids, void* stream) {
  const nvfp4_status st = logits_check(dtype, T, V, ld, scale);
  if (st != NVFP4_OK) return st;
  if (top_k < 0 || top_k > V) return NVFP4_ERR_INVALID_ARG;
  if (top_k > kMaxList) return NVFP4_ERR_UNSUPPORTED;
  if (T == 0) return NVFP4_OK;
  if (!aligned(logits, elt_bytes(dtype)) || !aligned(lse, 4) || !aligned_or_null(targets, 4) ||
      !aligned_or_null(logprob, 4) || !aligned_or_null(entropy, 4))
    return NVFP4_ERR_INVALID_ARG;
  if ((targets == nullptr) != (logprob == nullptr)) return NVFP4_ERR_INVALID_ARG;
  if (top_k > 0 && (!aligned(top_logprob, 4) || !aligned(top_ids, 4))) return NVFP4_ERR_INVALID_ARG;
  return from_cuda(launch_token_logprobs(logits, dtype, T, V, ld, targets, ignore_index, scale, top_k, logprob, lse,
                                         entropy, top_logprob, top_ids, static_cast<cudaStream_t>(stream)));
}

nvfp4_status token_logprobs_backward(const void* logits, nvfp4_act_dtype dtype, int64_t T, int64_t V, int64_t ld,
                                     const int32_t* targets, int32_t ignore_index, float scale, const float* lse,
                                     const float* entropy, const float* dlogprob, const float* dentropy,
                                     void* dlogits, int64_t ldd, void* stream) {
  const nvfp4_status st = logits_check(dtype, T, V, ld, scale);
  if (st != NVFP4_OK) return st;
  if (ldd < V) return NVFP4_ERR_INVALID_ARG;
  if (T == 0) return NVFP4_OK;
  const int e = elt_bytes(dtype);
  if (!aligned(logits, e) || !aligned(dlogits, e) || !aligned(lse, 4) || !aligned_or_null(targets, 4) ||
      !aligned_or_null(entropy, 4) || !aligned_or_null(dlogprob, 4) || !aligned_or_null(dentropy, 4))
    return NVFP4_ERR_INVALID_ARG;
  if (dlogprob != nullptr && targets == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (dentropy != nullptr && entropy == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (!same_or_disjoint(logits, ld, dlogits, ldd, T, V, e)) return NVFP4_ERR_INVALID_ARG;
  return from_cuda(launch_token_logprobs_backward(logits, dtype, T, V, ld, targets, ignore_index, scale, lse, entropy,
                                                  dlogprob, dentropy, dlogits, ldd,
                                                  static_cast<cudaStream_t>(stream)));
}

nvfp4_status distill_topk(const void* logits, nvfp4_act_dtype dtype, int64_t T, int64_t V, int64_t ld,
                          const int32_t* teacher_ids, const float* teacher_values, int32_t K, int tail, float scale,
                          float* loss, float* lse, void* stream) {
  const nvfp4_status st = logits_check(dtype, T, V, ld, scale);
  if (st != NVFP4_OK) return st;
  if (K <= 0) return NVFP4_ERR_INVALID_ARG;
  if (K > kMaxList) return NVFP4_ERR_UNSUPPORTED;
  if (T == 0) return NVFP4_OK;
  if (!aligned(logits, elt_bytes(dtype)) || !aligned(teacher_ids, 4) || !aligned(teacher_values, 4) ||
      !aligned(loss, 4) || !aligned_or_null(lse, 4))
    return NVFP4_ERR_INVALID_ARG;
  return from_cuda(launch_distill_topk(logits, dtype, T, V, ld, teacher_ids, teacher_values, K, tail != 0, scale,
                                       nullptr, loss, lse, nullptr, 0, static_cast<cudaStream_t>(stream)));
}

nvfp4_status distill_topk_backward(const void* logits, nvfp4_act_dtype dtype, int64_t T, int64_t V, int64_t ld,
                                   const int32_t* teacher_ids, const float* teacher_values, int32_t K, int tail,
                                   float scale, const float* dloss, float* loss, float* lse, void* dlogits,
                                   int64_t ldd, void* stream) {
  const nvfp4_status st = logits_check(dtype, T, V, ld, scale);
  if (st != NVFP4_OK) return st;
  if (K <= 0 || ldd < V) return NVFP4_ERR_INVALID_ARG;
  if (K > kMaxList) return NVFP4_ERR_UNSUPPORTED;
  if (T == 0) return NVFP4_OK;
  const int e = elt_bytes(dtype);
  if (!aligned(logits, e) || !aligned(dlogits, e) || !aligned(teacher_ids, 4) || !aligned(teacher_values, 4) ||
      !aligned(loss, 4) || !aligned_or_null(lse, 4) || !aligned_or_null(dloss, 4))
    return NVFP4_ERR_INVALID_ARG;
  if (!same_or_disjoint(logits, ld, dlogits, ldd, T, V, e)) return NVFP4_ERR_INVALID_ARG;
  return from_cuda(launch_distill_topk(logits, dtype, T, V, ld, teacher_ids, teacher_values, K, tail != 0, scale,
                                       dloss, loss, lse, dlogits, ldd, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
