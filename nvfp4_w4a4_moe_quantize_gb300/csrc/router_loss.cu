// The router's side of a learner's step: the balance loss with per-expert counts of every
// sequence, and the gradient of the router's logits.
//
// Of a sequence s with n counted tokens, p = softmax(logits) and c_e the times that expert e was
// chosen:   loss = E / (k n^2) sum_e c_e P_e,   P_e = sum_t p_te.   The counts are constants of the
// gradient, so with a_e = dloss E c_e / (k n^2) it is p_e (a_e - sum_j p_j a_j).  The routing weights
// add their own gradient: w_j = softmax over the chosen logits gives w_j (dw_j - sum_i w_i dw_i) at the
// chosen experts; plain probabilities w_j = p_j give w_j dw_j there, less p_e sum_i w_i dw_i everywhere.
//
// One warp holds one row: lane l the experts l, l + 32, ...
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "pdl.cuh"
#include "status.cuh"
#include "vocab.cuh"

namespace nvfp4 {
namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr uint32_t kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// First sequence that ends behind row r (S: none).  Sequences are offsets[0 .. S], not descending;
// without them all rows are sequence 0.
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, int64_t r, int64_t T) {
  if (offsets == nullptr) return r < T ? 0 : S;
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid + 1] > r) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// z becomes exp(z - max), its largest value the result's m, its sum the result's s.
template <int NV>
__device__ __forceinline__ void row_exp(float (&z)[NV], float& m, float& s) {
  m = z[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) m = fmaxf(m, z[i]);
  m = warp_max(m);
  const float mm = m == -INFINITY ? 0.f : m;   // every expert excluded
  s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    z[i] = ex2((z[i] - mm) * kLog2e);
    s += z[i];
  }
  s = warp_sum(s);
  m = mm;
}

struct BalanceArgs {
  const void* logits;
  int64_t T, ld;
  int E, k, S;
  const int32_t* ids;
  const int32_t* offsets;
  const uint8_t* valid;
  int64_t chunk;           // rows a CTA
  float* part_p;           // [slots][E]: slot chunk + sequence (one a pair that meets: either grows along the rows)
  int32_t* part_c;         // [slots][E]
  int32_t* part_n;         // [slots]
  float* loss;
  int32_t* counts;
  float* sums;
  int32_t* tokens;
  int* status;
};

template <typename T, int NV>
__global__ void __launch_bounds__(kThreads) balance_rows_kernel(const BalanceArgs a) {
  extern __shared__ float sm[];
  float* sm_p = sm;                                                    // [kWarps][E]
  int32_t* sm_c = reinterpret_cast<int32_t*>(sm + kWarps * a.E);       // [E]
  __shared__ int sm_n[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_sync();
  const int64_t r0 = blockIdx.x * a.chunk, r1 = min(a.T, r0 + a.chunk);
  for (int s = sequence_of(a.offsets, a.S, r0, a.T); s < a.S; ++s) {
    const int64_t lo = max(r0, a.offsets ? (int64_t)a.offsets[s] : 0), hi = min(r1, a.offsets ? (int64_t)a.offsets[s + 1] : a.T);
    if (lo >= r1) break;
    if (lo >= hi) continue;
    for (int e = threadIdx.x; e < a.E; e += kThreads) sm_c[e] = 0;
    __syncthreads();
    float p[NV];
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] = 0.f;
    for (int64_t r = lo + warp; r < hi; r += kWarps) {
      if (a.valid != nullptr && a.valid[r] == 0) continue;
      const T* row = static_cast<const T*>(a.logits) + r * a.ld;
      float z[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) z[i] = lane + 32 * i < a.E ? as_f32(row[lane + 32 * i]) : -INFINITY;
      const int id = lane < a.k ? a.ids[r * a.k + lane] : 0;
      float m, sum;
      row_exp<NV>(z, m, sum);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int i = 0; i < NV; ++i) p[i] = fmaf(z[i], inv, p[i]);
      if (lane < a.k) {
        if (id < 0 || id >= a.E) set_status(a.status, kStatusBadInput);
        else atomicAdd(&sm_c[id], 1);
      }
      ++n;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 32 * i < a.E) sm_p[warp * a.E + lane + 32 * i] = p[i];
    if (lane == 0) sm_n[warp] = n;
    __syncthreads();
    const int64_t slot = blockIdx.x + (int64_t)s;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      float t = 0.f;
      for (int w = 0; w < kWarps; ++w) t += sm_p[w * a.E + e];
      a.part_p[slot * a.E + e] = t;
      a.part_c[slot * a.E + e] = sm_c[e];
    }
    if (threadIdx.x == 0) {
      int t = 0;
      for (int w = 0; w < kWarps; ++w) t += sm_n[w];
      a.part_n[slot] = t;
    }
    __syncthreads();
  }
}

// One CTA a sequence: its slots' sums, each expert's in the order of the rows.
__global__ void __launch_bounds__(1024) balance_reduce_kernel(const BalanceArgs a) {
  __shared__ float sm_p[1024];
  __shared__ int32_t sm_c[1024];
  __shared__ float sm_w[32];
  __shared__ int sm_n;
  grid_dep_sync();
  const int s = blockIdx.x, tid = threadIdx.x;
  const int64_t lo = a.offsets ? (int64_t)a.offsets[s] : 0, hi = a.offsets ? (int64_t)a.offsets[s + 1] : a.T;
  const bool bad = lo < 0 || hi < lo || hi > a.T;
  const int64_t c0 = bad || lo == hi ? 0 : lo / a.chunk, c1 = bad || lo == hi ? 0 : (hi - 1) / a.chunk + 1;
  const int lanes = (a.E + 31) / 32 * 32, groups = 1024 / lanes;   // experts side by side, groups of slots
  const int e = tid % lanes, g = tid / lanes;
  float p = 0.f;
  int32_t c = 0;
  if (g < groups && e < a.E)
    for (int64_t i = c0 + g; i < c1; i += groups) {
      p += a.part_p[(i + s) * a.E + e];
      c += a.part_c[(i + s) * a.E + e];
    }
  sm_p[tid] = p;
  sm_c[tid] = c;
  if (tid < 32) {
    int n = 0;
    for (int64_t i = c0 + tid; i < c1; i += 32) n += a.part_n[i + s];
    n = __reduce_add_sync(kAll, n);
    if (tid == 0) sm_n = n;
  }
  __syncthreads();
  float cp = 0.f;
  if (tid < lanes && e < a.E) {
    for (int h = 1; h < groups; ++h) {
      p += sm_p[h * lanes + e];
      c += sm_c[h * lanes + e];
    }
    a.sums[(int64_t)s * a.E + e] = bad ? NAN : p;
    a.counts[(int64_t)s * a.E + e] = c;
    cp = static_cast<float>(c) * p;
  }
  cp = warp_sum(cp);
  if ((tid & 31) == 0) sm_w[tid >> 5] = cp;
  __syncthreads();
  if (tid < 32) {
    cp = warp_sum(sm_w[tid]);
    if (tid == 0) {
      const float n = static_cast<float>(sm_n);
      if (bad) set_status(a.status, kStatusBadInput);
      a.loss[s] = bad ? NAN : sm_n == 0 ? 0.f : static_cast<float>(a.E) / static_cast<float>(a.k) * (cp / n / n);
      a.tokens[s] = sm_n;
    }
  }
}

struct RouterBackwardArgs {
  const void* logits;
  int64_t T, ld;
  int E, k, S;
  const int32_t* ids;
  const float* dweights;   // nullable
  const float* dloss;      // nullable, with counts and tokens
  const int32_t* counts;
  const int32_t* tokens;
  const int32_t* offsets;
  const uint8_t* valid;
  void* dlogits;
  int64_t ldd;
  int64_t rows;            // rows a warp
  int* status;
};

constexpr int kBackWarps = 8;

template <typename T, int NV, bool kRenorm>
__global__ void __launch_bounds__(32 * kBackWarps) router_backward_kernel(const RouterBackwardArgs a) {
  extern __shared__ float sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* add = sm + warp * a.E;                                   // the chosen experts' part of the warp's row
  float* part = sm + kBackWarps * a.E + warp * 32;
  for (int e = lane; e < a.E; e += 32) add[e] = 0.f;
  __syncwarp();
  const int64_t r0 = ((int64_t)blockIdx.x * kBackWarps + warp) * a.rows, r1 = min(a.T, r0 + a.rows);
  if (r0 >= r1) return;
  const bool balance = a.dloss != nullptr;
  int s = a.S, held = -1;                                          // the row's sequence; that of al
  if (balance) s = sequence_of(a.offsets, a.S, r0, a.T);
  float al[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) al[i] = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const T* row = static_cast<const T*>(a.logits) + r * a.ld;
    float z[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) z[i] = lane + 32 * i < a.E ? as_f32(row[lane + 32 * i]) : -INFINITY;
    int id = -1;
    float dw = 0.f, zj = -INFINITY;
    if (a.dweights != nullptr && lane < a.k) {
      id = a.ids[r * a.k + lane];
      if (id < 0 || id >= a.E) {
        set_status(a.status, kStatusBadInput);
        id = -1;
      } else {
        dw = a.dweights[r * a.k + lane];
        zj = as_f32(row[id]);
      }
    }
    bool counted = false;
    if (balance) {
      if (a.offsets != nullptr)
        while (s < a.S && a.offsets[s + 1] <= r) ++s;
      counted = s < a.S && (a.offsets == nullptr || a.offsets[s] <= r) && (a.valid == nullptr || a.valid[r] != 0);
      if (counted && held != s) {
        const float n = static_cast<float>(max(a.tokens[s], 1));
        const float f = a.dloss[s] * (static_cast<float>(a.E) / static_cast<float>(a.k)) / n / n;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          al[i] = lane + 32 * i < a.E ? f * static_cast<float>(a.counts[(int64_t)s * a.E + lane + 32 * i]) : 0.f;
        held = s;
      }
    }
    float m, sum;
    row_exp<NV>(z, m, sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    float dot = 0.f;   // sum_e p_e of what every expert loses
    if (counted) {
#pragma unroll
      for (int i = 0; i < NV; ++i) dot = fmaf(z[i], al[i], dot);
      dot = warp_sum(dot) * inv;
    }
    if (a.dweights != nullptr) {
      float g;
      if (kRenorm) {
        const float mj = warp_max(zj);
        const float w = mj == -INFINITY ? 0.f : ex2((zj - mj) * kLog2e);
        const float ws = warp_sum(w);
        const float wn = ws == 0.f ? 0.f : w / ws;
        g = wn * (dw - warp_sum(wn * dw));
      } else {
        g = ex2((zj - m) * kLog2e) * inv * dw;
        dot += warp_sum(g);
      }
      // a chosen expert's part, once each: repeated ids add up in the order of their places
      part[lane] = g;
      __syncwarp();
      const uint32_t same = __match_any_sync(kAll, id);
      if (id >= 0 && lane == __ffs(same) - 1) {
        float t = 0.f;
        for (uint32_t b = same; b != 0; b &= b - 1) t += part[__ffs(b) - 1];
        add[id] = t;
      }
      __syncwarp();
    }
    T* out = static_cast<T*>(a.dlogits) + r * a.ldd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      if (e >= a.E) continue;
      float d = z[i] * inv * ((counted ? al[i] : 0.f) - dot);
      if (a.dweights != nullptr) {
        d += add[e];
        add[e] = 0.f;
      }
      put(out + e, d);
    }
    __syncwarp();
  }
}

template <typename F>
cudaError_t by_type_and_width(int dtype, int E, const F& f) {
  auto width = [&](auto t) {
    if (E <= 32) return f(t, std::integral_constant<int, 1>());
    if (E <= 64) return f(t, std::integral_constant<int, 2>());
    if (E <= 128) return f(t, std::integral_constant<int, 4>());
    if (E <= 256) return f(t, std::integral_constant<int, 8>());
    if (E <= 512) return f(t, std::integral_constant<int, 16>());
    return f(t, std::integral_constant<int, 32>());
  };
  if (dtype == kActBF16) return width(__nv_bfloat16());
  if (dtype == kActF16) return width(__half());
  return width(float());
}

}  // namespace

// Rows a CTA: one CTA an SM for the learner's batches.
static int64_t balance_chunk(int64_t T) {
  const int64_t c = (T + 151) / 152;
  return c < kWarps ? kWarps : c;
}

size_t balance_workspace(int64_t T, int64_t S, int64_t E) {
  const size_t chunk = (size_t)balance_chunk(T);
  const size_t slots = ((size_t)T + chunk - 1) / chunk + (size_t)S;
  return slots * ((size_t)E * 8 + 4);
}

cudaError_t launch_balance_loss(const void* logits, int dtype, int64_t T, int E, int64_t ld, const int32_t* ids, int k,
                                const int32_t* offsets, int S, const uint8_t* valid, float* loss, int32_t* counts,
                                float* sums, int32_t* tokens, void* workspace, cudaStream_t s) {
  BalanceArgs a{logits, T, ld, E, k, S, ids, offsets, valid, balance_chunk(T), nullptr, nullptr, nullptr,
                loss, counts, sums, tokens, device_status_ptr()};
  const int64_t chunks = (T + a.chunk - 1) / a.chunk, slots = chunks + S;
  a.part_p = static_cast<float*>(workspace);
  a.part_c = reinterpret_cast<int32_t*>(a.part_p + slots * E);
  a.part_n = a.part_c + slots * E;
  const size_t smem = (size_t)(kWarps + 1) * E * 4;
  const cudaError_t err = by_type_and_width(dtype, E, [&](auto t, auto nv) {
    auto* fn = balance_rows_kernel<decltype(t), decltype(nv)::value>;
    if (smem > 48 * 1024) {
      static std::atomic<bool> attr_set[64];
      const cudaError_t e = set_smem_attr_once(attr_set, (const void*)fn, (kWarps + 1) * 1024 * 4);
      if (e != cudaSuccess) return e;
    }
    return launch_pdl(false, fn, dim3((unsigned)chunks), dim3(kThreads), smem, s, a);
  });
  if (err != cudaSuccess) return err;
  return launch_pdl(true, balance_reduce_kernel, dim3((unsigned)S), dim3(1024), 0, s, a);
}

cudaError_t launch_router_backward(const void* logits, int dtype, int64_t T, int E, int64_t ld, const int32_t* ids,
                                   int k, const float* dweights, bool renorm, const float* dloss,
                                   const int32_t* counts, const int32_t* tokens, const int32_t* offsets, int S,
                                   const uint8_t* valid, void* dlogits, int64_t ldd, cudaStream_t s) {
  int64_t rows = (T + 152 * 64 - 1) / (152 * 64);   // 64 warps an SM
  RouterBackwardArgs a{logits, T, ld, E, k, S, ids, dweights, dloss, counts, tokens, offsets, valid, dlogits, ldd,
                       rows, device_status_ptr()};
  const int64_t ctas = (T + rows * kBackWarps - 1) / (rows * kBackWarps);
  const size_t smem = (size_t)kBackWarps * (E + 32) * 4;
  return by_type_and_width(dtype, E, [&](auto t, auto nv) {
    using El = decltype(t);
    constexpr int NV = decltype(nv)::value;
    if (renorm) router_backward_kernel<El, NV, true><<<(unsigned)ctas, 32 * kBackWarps, smem, s>>>(a);
    else router_backward_kernel<El, NV, false><<<(unsigned)ctas, 32 * kBackWarps, smem, s>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace nvfp4
