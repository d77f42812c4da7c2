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
  if (!(scale > 0.f) || !std::isfinite(scale * 2.f)) return NVFP4_ERR_INVALID_ARG;   // the kernels use scale log2(e)
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

nvfp4_status norm_check(nvfp4_act_dtype dtype, int64_t T, int64_t H, float eps) {
  if (!dtype_ok(dtype) || T < 0 || H <= 0 || !(eps > 0.f) || !std::isfinite(eps)) return NVFP4_ERR_INVALID_ARG;
  if (H > 8192 || T > ((int64_t)1 << 31) - 1) return NVFP4_ERR_UNSUPPORTED;
  return NVFP4_OK;
}
// No gate, one number a row, or gate_rows rows that each serve T / gate_rows rows.
bool gate_ok(const float* gate, int64_t gate_rows, int64_t T) {
  if (gate == nullptr) return gate_rows == 0;
  return gate_rows == 0 || (gate_rows > 0 && gate_rows <= 8192 && T % gate_rows == 0);
}

nvfp4_status head_check(nvfp4_act_dtype dtype, int64_t T, int64_t V, int64_t H, int64_t ldh, int64_t ldw, float scale) {
  if (!dtype_ok(dtype) || T < 0 || V <= 0 || H <= 0 || ldh < H || ldw < H) return NVFP4_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale * 2.f)) return NVFP4_ERR_INVALID_ARG;   // the kernels use scale log2(e)
  if (dtype == NVFP4_ACT_F32 || V > kMaxVocab || T > ((int64_t)1 << 20) || H > 16384 || H % 8 != 0 || ldh % 8 != 0 ||
      ldw % 8 != 0 || ldh > ((int64_t)1 << 32) || ldw > ((int64_t)1 << 32))
    return NVFP4_ERR_UNSUPPORTED;
  return NVFP4_OK;
}
// [n bytes from a] and [m bytes from b] have no byte in common.
bool disjoint(const void* a, int64_t n, const void* b, int64_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x + static_cast<uintptr_t>(n) <= y || y + static_cast<uintptr_t>(m) <= x;
}

nvfp4_status router_check(nvfp4_act_dtype dtype, int64_t T, int32_t E, int64_t ld, int32_t k, const int32_t* sequences,
                          int32_t S) {
  if (!dtype_ok(dtype) || T < 0 || E <= 0 || ld < E || k <= 0 || k > E || S <= 0) return NVFP4_ERR_INVALID_ARG;
  if ((sequences == nullptr && S != 1) || !aligned_or_null(sequences, 4)) return NVFP4_ERR_INVALID_ARG;
  if (E > 1024 || k > 32 || T > kMaxRows || S > (1 << 20)) return NVFP4_ERR_UNSUPPORTED;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

nvfp4_status head_logprobs(const void* hidden, int64_t ldh, const void* weight, int64_t ldw, nvfp4_act_dtype dtype,
                           int64_t T, int64_t V, int64_t H, const int32_t* targets, int32_t ignore_index, float scale,
                           float* logprob, float* lse, float* entropy, void* workspace, size_t workspace_bytes,
                           void* stream) {
  const nvfp4_status st = head_check(dtype, T, V, H, ldh, ldw, scale);
  if (st != NVFP4_OK) return st;
  if (T == 0) return NVFP4_OK;
  if (!aligned(hidden, 16) || !aligned(weight, 16) || !aligned(lse, 4) || !aligned_or_null(targets, 4) ||
      !aligned_or_null(logprob, 4) || !aligned_or_null(entropy, 4) || (targets == nullptr) != (logprob == nullptr))
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned(workspace, 16) || workspace_bytes < nvfp4_workspace_size(NVFP4_OP_HEAD_LOGPROBS, T, V, 0, H, 0))
    return NVFP4_ERR_WORKSPACE;
  return from_cuda(launch_head_logprobs(hidden, ldh, weight, ldw, dtype, T, V, H, targets, ignore_index, scale, logprob,
                                        lse, entropy, workspace, static_cast<cudaStream_t>(stream)));
}

nvfp4_status head_logprobs_backward(const void* hidden, int64_t ldh, const void* weight, int64_t ldw,
                                    nvfp4_act_dtype dtype, int64_t T, int64_t V, int64_t H, const int32_t* targets,
                                    int32_t ignore_index, float scale, const float* lse, const float* entropy,
                                    const float* dlogprob, const float* dentropy, void* dhidden, void* dweight,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  const nvfp4_status st = head_check(dtype, T, V, H, ldh, ldw, scale);
  if (st != NVFP4_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dweight != nullptr && !aligned(dweight, 16)) return NVFP4_ERR_INVALID_ARG;
  if (T == 0) return dweight == nullptr ? NVFP4_OK : from_cuda(cudaMemsetAsync(dweight, 0, 2 * (size_t)V * (size_t)H, s));
  if (dhidden == nullptr && dweight == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (dlogprob != nullptr && targets == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (dentropy != nullptr && entropy == nullptr) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(hidden, 16) || !aligned(weight, 16) || (dhidden != nullptr && !aligned(dhidden, 16)) ||
      !aligned(lse, 4) || !aligned_or_null(targets, 4) || !aligned_or_null(entropy, 4) ||
      !aligned_or_null(dlogprob, 4) || !aligned_or_null(dentropy, 4))
    return NVFP4_ERR_INVALID_ARG;
  const int64_t nh = 2 * ((T - 1) * ldh + H), nw = 2 * ((V - 1) * ldw + H), gh = 2 * T * H, gw = 2 * V * H;
  if ((dhidden != nullptr && (!disjoint(dhidden, gh, hidden, nh) || !disjoint(dhidden, gh, weight, nw))) ||
      (dweight != nullptr && (!disjoint(dweight, gw, hidden, nh) || !disjoint(dweight, gw, weight, nw))) ||
      (dhidden != nullptr && dweight != nullptr && !disjoint(dhidden, gh, dweight, gw)))
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned(workspace, 16) || workspace_bytes < nvfp4_workspace_size(NVFP4_OP_HEAD_LOGPROBS_BACKWARD, T, V, 0, H, 0))
    return NVFP4_ERR_WORKSPACE;
  return from_cuda(launch_head_logprobs_backward(hidden, ldh, weight, ldw, dtype, T, V, H, targets, ignore_index, scale,
                                                 lse, entropy, dlogprob, dentropy, dhidden, dweight, workspace, s));
}

nvfp4_status moe_balance_loss(const void* logits, nvfp4_act_dtype dtype, int64_t T, int32_t E, int64_t ld,
                              const int32_t* ids, int32_t k, const int32_t* sequences, int32_t S,
                              const uint8_t* valid, float* loss, int32_t* counts, float* prob_sums, int32_t* tokens,
                              void* workspace, size_t workspace_bytes, void* stream) {
  const nvfp4_status st = router_check(dtype, T, E, ld, k, sequences, S);
  if (st != NVFP4_OK) return st;
  if (!aligned(loss, 4) || !aligned(counts, 4) || !aligned(prob_sums, 4) || !aligned(tokens, 4))
    return NVFP4_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    const size_t n = 4 * (size_t)S;
    cudaError_t err = cudaMemsetAsync(loss, 0, n, s);
    if (err == cudaSuccess) err = cudaMemsetAsync(tokens, 0, n, s);
    if (err == cudaSuccess) err = cudaMemsetAsync(counts, 0, n * (size_t)E, s);
    if (err == cudaSuccess) err = cudaMemsetAsync(prob_sums, 0, n * (size_t)E, s);
    return from_cuda(err);
  }
  if (!aligned(logits, elt_bytes(dtype)) || !aligned(ids, 4)) return NVFP4_ERR_INVALID_ARG;
  const size_t need = nvfp4_workspace_size(NVFP4_OP_BALANCE_LOSS, T, S, E, 0, 0);
  if (need > 0 && (!aligned(workspace, 16) || workspace_bytes < need)) return NVFP4_ERR_WORKSPACE;
  return from_cuda(launch_balance_loss(logits, dtype, T, E, ld, ids, k, sequences, S, valid, loss, counts, prob_sums,
                                       tokens, workspace, s));
}

nvfp4_status moe_router_backward(const void* logits, nvfp4_act_dtype dtype, int64_t T, int32_t E, int64_t ld,
                                 const int32_t* ids, int32_t k, const float* dweights, int renormalize,
                                 const float* dloss, const int32_t* counts, const int32_t* tokens,
                                 const int32_t* sequences, int32_t S, const uint8_t* valid, void* dlogits,
                                 int64_t ldd, void* stream) {
  const nvfp4_status st = router_check(dtype, T, E, ld, k, sequences, S);
  if (st != NVFP4_OK) return st;
  if (ldd < E) return NVFP4_ERR_INVALID_ARG;
  if (T == 0) return NVFP4_OK;
  if (dweights == nullptr && dloss == nullptr) return NVFP4_ERR_INVALID_ARG;
  const int e = elt_bytes(dtype);
  if (!aligned(logits, e) || !aligned(dlogits, e)) return NVFP4_ERR_INVALID_ARG;
  if (dweights != nullptr && (!aligned(dweights, 4) || !aligned(ids, 4))) return NVFP4_ERR_INVALID_ARG;
  if (dloss != nullptr && (!aligned(dloss, 4) || !aligned(counts, 4) || !aligned(tokens, 4))) return NVFP4_ERR_INVALID_ARG;
  if (!same_or_disjoint(logits, ld, dlogits, ldd, T, E, e)) return NVFP4_ERR_INVALID_ARG;
  return from_cuda(launch_router_backward(logits, dtype, T, E, ld, ids, k, dweights, renormalize != 0, dloss, counts,
                                          tokens, sequences, S, valid, dlogits, ldd,
                                          static_cast<cudaStream_t>(stream)));
}

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

nvfp4_status moe_norm_in(const void* x, int64_t ldx, nvfp4_act_dtype dtype, int64_t T, int64_t H, const float* weight,
                         float eps, void* n, float* rstd, void* stream) {
  const nvfp4_status st = norm_check(dtype, T, H, eps);
  if (st != NVFP4_OK) return st;
  if (ldx < H) return NVFP4_ERR_INVALID_ARG;
  if (T == 0) return NVFP4_OK;
  const int e = elt_bytes(dtype);
  if (!aligned(x, e) || !aligned(n, e) || !aligned(weight, 4) || !aligned(rstd, 4)) return NVFP4_ERR_INVALID_ARG;
  return from_cuda(launch_block_norm(x, ldx, nullptr, 0, dtype, T, H, nullptr, nullptr, 0, 1.f, weight, eps, nullptr, n,
                                     nullptr, rstd, static_cast<cudaStream_t>(stream)));
}

nvfp4_status moe_norm_in_backward(const void* dn, int64_t lddn, const void* dresidual, int64_t lddr, const void* x,
                                  int64_t ldx, const float* rstd, nvfp4_act_dtype dtype, int64_t T, int64_t H,
                                  const float* weight, void* dx, float* dweight, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  const nvfp4_status st = norm_check(dtype, T, H, 1.f);
  if (st != NVFP4_OK) return st;
  if (lddn < H || ldx < H || (dresidual != nullptr && lddr < H)) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(dweight, 4)) return NVFP4_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) return from_cuda(cudaMemsetAsync(dweight, 0, 4 * (size_t)H, s));
  const int e = elt_bytes(dtype);
  if (!aligned(dn, e) || !aligned_or_null(dresidual, e) || !aligned(x, e) || !aligned(dx, e) || !aligned(rstd, 4) ||
      !aligned(weight, 4))
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned(workspace, 16) || workspace_bytes < nvfp4_workspace_size(NVFP4_OP_NORM_BACKWARD, T, 0, 0, H, 0))
    return NVFP4_ERR_WORKSPACE;
  return from_cuda(launch_block_norm_backward(dresidual, lddr, dn, lddn, x, ldx, nullptr, 0, dtype, T, H, nullptr, rstd,
                                              nullptr, nullptr, 0, 1.f, weight, dx, nullptr, nullptr, nullptr, dweight,
                                              static_cast<float*>(workspace), s));
}

nvfp4_status moe_norm_out(const void* x, int64_t ldx, const void* y, int64_t ldy, nvfp4_act_dtype dtype, int64_t T,
                          int64_t H, const float* weight, const float* gate, int64_t gate_rows, float residual_scale,
                          const float* next_weight, float eps, void* r, void* n, float* rstd_y, float* rstd_r,
                          void* stream) {
  const nvfp4_status st = norm_check(dtype, T, H, eps);
  if (st != NVFP4_OK) return st;
  if (ldx < H || ldy < H || !gate_ok(gate, gate_rows, T) || !std::isfinite(residual_scale))
    return NVFP4_ERR_INVALID_ARG;
  if (T == 0) return NVFP4_OK;
  const int e = elt_bytes(dtype);
  if (!aligned(x, e) || !aligned(y, e) || !aligned(r, e) || !aligned(weight, 4) || !aligned(rstd_y, 4) ||
      !aligned_or_null(gate, 4))
    return NVFP4_ERR_INVALID_ARG;
  if (next_weight != nullptr && (!aligned(next_weight, 4) || !aligned(n, e) || !aligned(rstd_r, 4)))
    return NVFP4_ERR_INVALID_ARG;
  return from_cuda(launch_block_norm(x, ldx, y, ldy, dtype, T, H, weight, gate, gate_rows, residual_scale, next_weight,
                                     eps, r, n, rstd_y, rstd_r, static_cast<cudaStream_t>(stream)));
}

nvfp4_status moe_norm_out_backward(const void* dr, int64_t lddr, const void* dn, int64_t lddn, const void* r,
                                   int64_t ldr, const void* y, int64_t ldy, const float* rstd_y, const float* rstd_r,
                                   nvfp4_act_dtype dtype, int64_t T, int64_t H, const float* weight,
                                   const float* gate, int64_t gate_rows, float residual_scale,
                                   const float* next_weight, void* dx, void* dy, float* dweight, float* dgate,
                                   float* dnext_weight, void* workspace, size_t workspace_bytes, void* stream) {
  const nvfp4_status st = norm_check(dtype, T, H, 1.f);
  if (st != NVFP4_OK) return st;
  if (ldy < H || (dr != nullptr && lddr < H) || !gate_ok(gate, gate_rows, T) || !std::isfinite(residual_scale))
    return NVFP4_ERR_INVALID_ARG;
  const bool next = next_weight != nullptr;
  if (next && (lddn < H || ldr < H)) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(dweight, 4) || (gate != nullptr && !aligned(dgate, 4)) || (next && !aligned(dnext_weight, 4)))
    return NVFP4_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    cudaError_t err = cudaMemsetAsync(dweight, 0, 4 * (size_t)H, s);
    if (err == cudaSuccess && next) err = cudaMemsetAsync(dnext_weight, 0, 4 * (size_t)H, s);
    if (err == cudaSuccess && gate_rows > 0) err = cudaMemsetAsync(dgate, 0, 4 * (size_t)(gate_rows * H), s);
    return from_cuda(err);
  }
  const int e = elt_bytes(dtype);
  if (!aligned(y, e) || !aligned(dx, e) || !aligned(dy, e) || !aligned(rstd_y, 4) || !aligned(weight, 4) ||
      !aligned_or_null(gate, 4) || !aligned_or_null(dr, e))
    return NVFP4_ERR_INVALID_ARG;
  if (next ? !aligned(dn, e) || !aligned(r, e) || !aligned(rstd_r, 4) || !aligned(next_weight, 4) : dr == nullptr)
    return NVFP4_ERR_INVALID_ARG;
  if (!aligned(workspace, 16) || workspace_bytes < nvfp4_workspace_size(NVFP4_OP_NORM_BACKWARD, T, gate_rows, 0, H, 0))
    return NVFP4_ERR_WORKSPACE;
  return from_cuda(launch_block_norm_backward(dr, lddr, next ? dn : nullptr, lddn, r, ldr, y, ldy, dtype, T, H, rstd_y,
                                              rstd_r, weight, gate, gate_rows, residual_scale, next_weight, dx, dy,
                                              dweight, dgate, dnext_weight, static_cast<float*>(workspace), s));
}

}  // extern "C"
