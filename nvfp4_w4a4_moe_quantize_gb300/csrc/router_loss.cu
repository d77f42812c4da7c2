// The router's side of a learner's step: the balance loss with per-expert counts of every
// sequence, and the gradient of the router's logits.
//
// Of a sequence s with n counted tokens, p = softmax(logits) and c_e the times that expert e was
// chosen:   loss = E / (k n^2) sum_e c_e P_e,   P_e = sum_t p_te.   The counts are constants of the
// gradient, so with a_e = dloss E c_e / (k n^2) it is p_e (a_e - sum_j p_j a_j).  The routing weights
// add their own gradient: w_j = softmax over the chosen logits gives w_j (dw_j - sum_i w_i dw_i) at the
// chosen experts; plain probabilities w_j = p_j give w_j dw_j there, less p_e sum_i w_i dw_i everywhere.
//
// A warp holds a row: lane l the experts l, l + 32, ...; it works on several rows at once, since a row's loads
// and sums over the lanes are a long chain of little work (one row at a time measured 15 and 22 us for the losses'
// and the gradient's kernel at 32768 x 128 float32 logits, whose traffic takes 3 and 5; as it is 10 and 18).  What
// bounds them is this layout's instructions: at 128 experts a lane has four numbers, and a sum over the lanes takes five
// steps.  Spills: the gradient's kernel at 65 to 128 experts 44-52 bytes stored and 16-92 loaded at the 64 registers that
// four CTAs an SM leave, at 33 to 64 up to 8 and 28; the losses' above 512 experts 152-216 each way.
#include <algorithm>
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

constexpr int kWarps = 32, kThreads = 32 * kWarps;
constexpr uint32_t kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

template <int kFirst = 16, int RB>
__device__ __forceinline__ void warp_max(float (&v)[RB]) {
#pragma unroll
  for (int d = kFirst; d > 0; d >>= 1)
#pragma unroll
    for (int b = 0; b < RB; ++b) v[b] = fmaxf(v[b], __shfl_xor_sync(kAll, v[b], d));
}
// (over groups of 2 kFirst neighbouring lanes)
template <int kFirst = 16, int RB>
__device__ __forceinline__ void warp_sum(float (&v)[RB]) {
#pragma unroll
  for (int d = kFirst; d > 0; d >>= 1)
#pragma unroll
    for (int b = 0; b < RB; ++b) v[b] += __shfl_xor_sync(kAll, v[b], d);
}
__device__ __forceinline__ float warp_sum(float v) {
  float w[1] = {v};
  warp_sum(w);
  return w[0];
}

// Rows that a warp works on at once.
__host__ __device__ constexpr int rows_at_once(int nv) { return nv <= 4 ? 4 : nv <= 8 ? 2 : 1; }

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

// Of every row: z becomes exp(z - max), m the max (0 where every expert is excluded), inv 1 over the sum (0 there).
template <int RB, int NV>
__device__ __forceinline__ void rows_exp(float (&z)[RB][NV], float (&m)[RB], float (&inv)[RB]) {
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    m[b] = z[b][0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m[b] = fmaxf(m[b], z[b][i]);
  }
  warp_max(m);
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    if (m[b] == -INFINITY) m[b] = 0.f;
    inv[b] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      z[b][i] = ex2((z[b][i] - m[b]) * kLog2e);
      inv[b] += z[b][i];
    }
  }
  warp_sum(inv);
#pragma unroll
  for (int b = 0; b < RB; ++b) inv[b] = inv[b] == 0.f ? 0.f : 1.f / inv[b];
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
  int32_t* part_bad;       // [chunks]: whether the list of sequences descends in a CTA's part of it
  float* loss;
  int32_t* counts;
  float* sums;
  int32_t* tokens;
  int* status;
};

// The loss of a sequence from its counts c and sums p, an expert a thread (threads beyond E give 0).
__device__ __forceinline__ float balance_of(int E, int k, int32_t c, float p, int n, float* sm_w) {
  float cp = warp_sum(static_cast<float>(c) * p);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) sm_w[warp] = cp;
  __syncthreads();
  cp = warp_sum(sm_w[lane]);
  const float f = static_cast<float>(n);
  return n == 0 ? 0.f : static_cast<float>(E) / static_cast<float>(k) * (cp / f / f);
}

// kWhole: one CTA, one sequence: the results at once.
template <typename T, int NV, bool kWhole>
__global__ void __launch_bounds__(kThreads) balance_rows_kernel(const BalanceArgs a) {
  constexpr int RB = rows_at_once(NV);
  extern __shared__ float sm[];
  float* sm_p = sm;                                                    // [kWarps][E]
  int32_t* sm_c = reinterpret_cast<int32_t*>(sm + kWarps * a.E);       // [E]
  __shared__ int sm_n[kWarps];
  __shared__ float sm_w[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_sync();
  const int64_t r0 = blockIdx.x * a.chunk, r1 = min(a.T, r0 + a.chunk);
  bool descends = false;
  if (!kWhole && a.offsets != nullptr)
    for (int s = blockIdx.x * kThreads + threadIdx.x; s < a.S; s += gridDim.x * kThreads)
      descends |= a.offsets[s + 1] < a.offsets[s];
  // A list that descends: a single CTA takes every sequence for itself.  Several need the order for their search and
  // their slots; they give no results, and no row is read twice on the way to that.
  const bool each = !kWhole && gridDim.x == 1 && __syncthreads_or(descends);
  int64_t done = r0;
  for (int s = kWhole || each ? 0 : sequence_of(a.offsets, a.S, r0, a.T); s < a.S; ++s) {
    const int64_t lo = max(each ? r0 : done, a.offsets ? (int64_t)a.offsets[s] : 0);
    const int64_t hi = min(r1, a.offsets ? (int64_t)a.offsets[s + 1] : a.T);
    if (!kWhole) {
      if (lo >= r1 && !each) break;
      if (lo >= hi) continue;
      done = hi;
    }
    for (int e = threadIdx.x; e < a.E; e += kThreads) sm_c[e] = 0;
    __syncthreads();
    float p[NV];
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] = 0.f;
    for (int64_t r = lo + warp; r < hi; r += kWarps * RB) {
      float z[RB][NV], m[RB], inv[RB];
      int id[RB];
      bool on[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const int64_t t = r + b * kWarps;
        on[b] = t < hi && (a.valid == nullptr || a.valid[t] != 0);
        const T* row = static_cast<const T*>(a.logits) + t * a.ld;
#pragma unroll
        for (int i = 0; i < NV; ++i) z[b][i] = on[b] && lane + 32 * i < a.E ? as_f32(row[lane + 32 * i]) : -INFINITY;
        id[b] = on[b] && lane < a.k ? a.ids[t * a.k + lane] : 0;
      }
      rows_exp(z, m, inv);
#pragma unroll
      for (int b = 0; b < RB; ++b) {
#pragma unroll
        for (int i = 0; i < NV; ++i) p[i] = fmaf(z[b][i], inv[b], p[i]);
        if (on[b] && lane < a.k) {
          if (id[b] < 0 || id[b] >= a.E) set_status(a.status, kStatusBadInput);
          else atomicAdd(&sm_c[id[b]], 1);
        }
        n += on[b];
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 32 * i < a.E) sm_p[warp * a.E + lane + 32 * i] = p[i];
    if (lane == 0) sm_n[warp] = n;
    __syncthreads();
    n = __reduce_add_sync(kAll, sm_n[lane]);
    const int e = threadIdx.x;   // E <= kThreads
    float t = 0.f;
    if (e < a.E)
      for (int w = 0; w < kWarps; ++w) t += sm_p[w * a.E + e];
    if (kWhole) {
      const float loss = balance_of(a.E, a.k, e < a.E ? sm_c[e] : 0, t, n, sm_w);
      const bool bad = a.offsets != nullptr && (a.offsets[0] < 0 || a.offsets[1] < a.offsets[0] || a.offsets[1] > a.T);
      if (e < a.E) {
        a.sums[e] = bad ? NAN : t;
        a.counts[e] = bad ? 0 : sm_c[e];
      }
      if (threadIdx.x == 0) {
        if (bad) set_status(a.status, kStatusBadInput);
        a.loss[0] = bad ? NAN : loss;
        a.tokens[0] = bad ? 0 : n;
      }
      return;
    }
    const int64_t slot = blockIdx.x + (int64_t)s;
    if (e < a.E) {
      a.part_p[slot * a.E + e] = t;
      a.part_c[slot * a.E + e] = sm_c[e];
    }
    if (threadIdx.x == 0) a.part_n[slot] = n;
    __syncthreads();
  }
  if (!kWhole) {
    descends = __syncthreads_or(descends) && !each;
    if (threadIdx.x == 0) a.part_bad[blockIdx.x] = descends;
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
  bool bad = lo < 0 || hi < lo || hi > a.T;
  const int chunks = static_cast<int>((a.T + a.chunk - 1) / a.chunk);   // at most 152
  const bool descends = tid < chunks && a.part_bad[tid] != 0;
  const int64_t c0 = bad || lo == hi ? 0 : lo / a.chunk, c1 = bad || lo == hi ? 0 : (hi - 1) / a.chunk + 1;
  const int lanes = (a.E + 31) / 32 * 32, groups = 1024 / lanes;   // experts side by side, groups of slots
  const int e = tid % lanes, g = tid / lanes;
  float p = 0.f;
  int32_t c = 0;
  if (g < groups && e < a.E) {
    for (int64_t i0 = c0 + g; i0 < c1; i0 += 8 * groups) {   // eight loads of each on their way
      float pi[8];
      int32_t ci[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t i = i0 + j * groups;
        pi[j] = i < c1 ? a.part_p[(i + s) * a.E + e] : 0.f;
        ci[j] = i < c1 ? a.part_c[(i + s) * a.E + e] : 0;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) p += pi[j], c += ci[j];
    }
  }
  sm_p[tid] = p;
  sm_c[tid] = c;
  if (tid < 32) {
    int n = 0;
#pragma unroll 4
    for (int64_t i = c0 + tid; i < c1; i += 32) n += a.part_n[i + s];
    n = __reduce_add_sync(kAll, n);
    if (tid == 0) sm_n = n;
  }
  bad |= __syncthreads_or(descends) != 0;
  const bool mine = tid < lanes && e < a.E;
  if (mine) {
    for (int h = 1; h < groups; ++h) {
      p += sm_p[h * lanes + e];
      c += sm_c[h * lanes + e];
    }
    a.sums[(int64_t)s * a.E + e] = bad ? NAN : p;
    a.counts[(int64_t)s * a.E + e] = bad ? 0 : c;
  }
  const float loss = balance_of(a.E, a.k, mine ? c : 0, mine ? p : 0.f, sm_n, sm_w);
  if (tid == 0) {
    if (bad) set_status(a.status, kStatusBadInput);
    a.loss[s] = bad ? NAN : loss;
    a.tokens[s] = bad ? 0 : sm_n;
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

// kFew: at most 8 experts are chosen, and sums over them take 8 lanes.
template <typename T, int NV, bool kRenorm, bool kFew>
__global__ void __launch_bounds__(32 * kBackWarps, NV <= 4 ? 4 : 1) router_backward_kernel(const RouterBackwardArgs a) {
  constexpr int RB = rows_at_once(NV), kChosen = kFew ? 4 : 16;
  extern __shared__ float sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* add = sm + warp * RB * a.E;                              // the chosen experts' part of each row
  float* part = sm + kBackWarps * RB * a.E + warp * 32;
  if (a.dweights != nullptr)
    for (int e = lane; e < RB * a.E; e += 32) add[e] = 0.f;
  __syncwarp();
  const int64_t r0 = ((int64_t)blockIdx.x * kBackWarps + warp) * a.rows, r1 = min(a.T, r0 + a.rows);
  if (r0 >= r1) return;
  const bool balance = a.dloss != nullptr;
  int s = a.S, held = -1;                                          // the next row's sequence; that of al
  if (balance) s = sequence_of(a.offsets, a.S, r0, a.T);
  float al[NV];
  auto hold = [&](int q) {                                         // al = what sequence q's tokens gain
    if (q == held) return;
    const float n = static_cast<float>(max(a.tokens[q], 1));
    const float f = a.dloss[q] * (static_cast<float>(a.E) / static_cast<float>(a.k)) / n / n;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      al[i] = lane + 32 * i < a.E ? f * static_cast<float>(a.counts[(int64_t)q * a.E + lane + 32 * i]) : 0.f;
    held = q;
  };
  for (int64_t r = r0; r < r1; r += RB) {
    float z[RB][NV], m[RB], inv[RB], dw[RB], zj[RB], dot[RB];
    int id[RB], seq[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int64_t t = r + b;
      const bool on = t < r1;
      const T* row = static_cast<const T*>(a.logits) + t * a.ld;
#pragma unroll
      for (int i = 0; i < NV; ++i) z[b][i] = on && lane + 32 * i < a.E ? as_f32(row[lane + 32 * i]) : -INFINITY;
      const bool chosen = on && a.dweights != nullptr && lane < a.k;
      id[b] = chosen ? a.ids[t * a.k + lane] : -1;
      dw[b] = chosen ? a.dweights[t * a.k + lane] : 0.f;
      if (chosen && (id[b] < 0 || id[b] >= a.E)) {
        set_status(a.status, kStatusBadInput);
        id[b] = -1;
        dw[b] = 0.f;
      }
      seq[b] = -1;                                                 // the balance loss does not reach it
      if (balance && on) {
        if (a.offsets != nullptr)
          while (s < a.S && a.offsets[s + 1] <= t) ++s;
        if (s < a.S && (a.offsets == nullptr || a.offsets[s] <= t) && (a.valid == nullptr || a.valid[t] != 0)) seq[b] = s;
      }
      if (a.dweights == nullptr && seq[b] < 0) {                   // its gradient is 0, whatever it holds
#pragma unroll
        for (int i = 0; i < NV; ++i) z[b][i] = -INFINITY;
      }
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) {                                 // the chosen experts' logits
      zj[b] = -INFINITY;
      if (a.dweights == nullptr) continue;
      if (NV <= 8) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const float v = __shfl_sync(kAll, z[b][i], id[b] & 31);
          if (id[b] >> 5 == i) zj[b] = v;
        }
      } else if (id[b] >= 0) {
        zj[b] = as_f32(static_cast<const T*>(a.logits)[(r + b) * a.ld + id[b]]);
      }
    }
    rows_exp(z, m, inv);
#pragma unroll
    for (int b = 0; b < RB; ++b) {   // dot: sum_e p_e of what every expert gains
      dot[b] = 0.f;
      if (seq[b] < 0) continue;
      hold(seq[b]);
#pragma unroll
      for (int i = 0; i < NV; ++i) dot[b] = fmaf(z[b][i], al[i], dot[b]);
    }
    if (balance) {
      warp_sum(dot);
#pragma unroll
      for (int b = 0; b < RB; ++b) dot[b] *= inv[b];
    }
    if (a.dweights != nullptr) {
      float g[RB], w[RB];
      if (kRenorm) {
        float mj[RB], ws[RB], wd[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) mj[b] = zj[b];
        warp_max<kChosen>(mj);
#pragma unroll
        for (int b = 0; b < RB; ++b) ws[b] = w[b] = mj[b] == -INFINITY ? 0.f : ex2((zj[b] - mj[b]) * kLog2e);
        warp_sum<kChosen>(ws);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          w[b] = ws[b] == 0.f ? 0.f : w[b] / ws[b];
          wd[b] = w[b] * dw[b];
        }
        warp_sum<kChosen>(wd);
#pragma unroll
        for (int b = 0; b < RB; ++b) g[b] = w[b] * (dw[b] - wd[b]);
      } else {
#pragma unroll
        for (int b = 0; b < RB; ++b) w[b] = g[b] = ex2((zj[b] - m[b]) * kLog2e) * inv[b] * dw[b];
        warp_sum(w);
#pragma unroll
        for (int b = 0; b < RB; ++b) dot[b] += w[b];
      }
      // a chosen expert's part, once each: an id is alone if its place still has the lane that wrote there
#pragma unroll
      for (int b = 0; b < RB; ++b)
        if (id[b] >= 0) add[b * a.E + id[b]] = __int_as_float(lane);
      __syncwarp();
      bool twice = false;
#pragma unroll
      for (int b = 0; b < RB; ++b) twice |= id[b] >= 0 && __float_as_int(add[b * a.E + id[b]]) != lane;
      if (__any_sync(kAll, twice)) {
        // repeated ids add up in the order of their places
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          part[lane] = g[b];
          __syncwarp();
          const uint32_t same = __match_any_sync(kAll, id[b]);
          float t = 0.f;
          for (uint32_t q = same; q != 0; q &= q - 1) t += part[__ffs(q) - 1];
          g[b] = t;
          __syncwarp();
        }
      }
#pragma unroll
      for (int b = 0; b < RB; ++b)
        if (id[b] >= 0) add[b * a.E + id[b]] = g[b];   // repeated ids write the same sum
      __syncwarp();
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      if (r + b >= r1) break;
      T* out = static_cast<T*>(a.dlogits) + (r + b) * a.ldd;
      if (seq[b] >= 0) hold(seq[b]);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        if (e >= a.E) continue;
        float d = z[b][i] * inv[b] * ((seq[b] >= 0 ? al[i] : 0.f) - dot[b]);
        if (a.dweights != nullptr) {
          d += add[b * a.E + e];
          add[b * a.E + e] = 0.f;
        }
        put(out + e, d);
      }
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
// One CTA takes them all, a group of rows or two a warp: no partial results and no second kernel.  On the device,
// one kernel / two: 256 x 8 6.3 / 7.3 us, 256 x 128 7.3 / 8.1, 32 x 1024 9.0 / 10.4; 512 x 128 11.0 / 8.5, 64 x 1024
// 12.6 / 10.3.
static bool balance_whole(int64_t T, int64_t S, int64_t E) {
  return S == 1 && T <= kWarps * rows_at_once((int)((E + 31) / 32)) * (E <= 256 ? 2 : 1);
}

size_t balance_workspace(int64_t T, int64_t S, int64_t E) {
  if (balance_whole(T, S, E)) return 0;
  // (the most that this T or a smaller one has: a workspace for the largest batch serves the others)
  const size_t chunks = std::min<size_t>(((size_t)T + kWarps - 1) / kWarps, 152), slots = chunks + (size_t)S;
  return slots * ((size_t)E * 8 + 4) + chunks * 4;
}

cudaError_t launch_balance_loss(const void* logits, int dtype, int64_t T, int E, int64_t ld, const int32_t* ids, int k,
                                const int32_t* offsets, int S, const uint8_t* valid, float* loss, int32_t* counts,
                                float* sums, int32_t* tokens, void* workspace, cudaStream_t s) {
  BalanceArgs a{logits, T, ld, E, k, S, ids, offsets, valid, balance_chunk(T), nullptr, nullptr, nullptr, nullptr,
                loss, counts, sums, tokens, device_status_ptr()};
  const int64_t chunks = (T + a.chunk - 1) / a.chunk, slots = chunks + S;
  a.part_p = static_cast<float*>(workspace);
  a.part_c = reinterpret_cast<int32_t*>(a.part_p + slots * E);
  a.part_n = a.part_c + slots * E;
  a.part_bad = a.part_n + slots;
  const size_t smem = (size_t)(kWarps + 1) * E * 4;
  const bool whole = balance_whole(T, S, E);
  if (whole) a.chunk = T;
  const cudaError_t err = by_type_and_width(dtype, E, [&](auto t, auto nv) {
    using El = decltype(t);
    constexpr int NV = decltype(nv)::value;
    auto* fn = whole ? balance_rows_kernel<El, NV, true> : balance_rows_kernel<El, NV, false>;
    if (smem > 47 * 1024) {   // (48 KB are free to every launch; the kernel's static 256 bytes count as well)
      static std::atomic<bool> attr_set[2][64];
      const cudaError_t e = set_smem_attr_once(attr_set[whole], (const void*)fn, (kWarps + 1) * 1024 * 4);
      if (e != cudaSuccess) return e;
    }
    return launch_pdl(false, fn, dim3(whole ? 1u : (unsigned)chunks), dim3(kThreads), smem, s, a);
  });
  if (err != cudaSuccess || whole) return err;
  return launch_pdl(true, balance_reduce_kernel, dim3((unsigned)S), dim3(1024), 0, s, a);
}

cudaError_t launch_router_backward(const void* logits, int dtype, int64_t T, int E, int64_t ld, const int32_t* ids,
                                   int k, const float* dweights, bool renorm, const float* dloss,
                                   const int32_t* counts, const int32_t* tokens, const int32_t* offsets, int S,
                                   const uint8_t* valid, void* dlogits, int64_t ldd, cudaStream_t s) {
  // 64 warps an SM, whole groups of the rows that a warp takes at once
  const int at_once = rows_at_once((E + 31) / 32);
  const int64_t rows = ((T + 152 * 64 - 1) / (152 * 64) + at_once - 1) / at_once * at_once;
  RouterBackwardArgs a{logits, T, ld, E, k, S, ids, dweights, dloss, counts, tokens, offsets, valid, dlogits, ldd,
                       rows, device_status_ptr()};
  const int64_t ctas = (T + rows * kBackWarps - 1) / (rows * kBackWarps);
  return by_type_and_width(dtype, E, [&](auto t, auto nv) {
    using El = decltype(t);
    constexpr int NV = decltype(nv)::value;
    const size_t smem = (size_t)kBackWarps * (rows_at_once(NV) * E + 32) * 4;   // at most 33 KB
    auto* fn = renorm ? (k <= 8 ? router_backward_kernel<El, NV, true, true> : router_backward_kernel<El, NV, true, false>)
                      : router_backward_kernel<El, NV, false, false>;
    fn<<<(unsigned)ctas, 32 * kBackWarps, smem, s>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace nvfp4
