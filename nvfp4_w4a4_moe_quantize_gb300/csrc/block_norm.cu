// RMS norms before and after the expert block, fused with the block's gate and the residual's
// scale, and their backward.
//
//   n = x rstd(x) w                                    rstd(x) = 1 / sqrt(mean(x^2) + eps)
//   r = a x + gate (y rstd(y) w);   n' = r rstd(r) w'  (r as it is stored)
//
// A row stays in registers between its reductions: x and y are read once, r and n' written
// once.  A row belongs to a group of G threads, G a function of H alone, two chunks of 8
// elements a thread; sums run in that fixed order, so a row's bits do not depend on the batch.
// Backward: a CTA takes a range of rows of one gate row and keeps the column sums of the
// weights' and gate's gradients in registers; the ranges' sums are added by a second kernel
// in a fixed order (no atomics).
#include "launch.h"
#include "vocab.cuh"

namespace nvfp4 {
namespace {

constexpr int kChunks = 2;        // chunks of 8 elements a thread
constexpr int kNormThreads = 256; // at least; a group of 512 is a CTA of its own

// Threads a row: the smallest power of two >= 32 that holds H.
inline int group_threads(int64_t H) {
  int g = 32;
  while (g * kChunks * 8 < H) g *= 2;
  return g;
}

// 8 values as pairs: elements [e, e + 8) of a row, zero beyond it.  kVec: the rows are 16-byte
// aligned and whole chunks; else element by element.
struct Eight {
  F2 p[4];
};
template <typename E, bool kVec>
__device__ __forceinline__ Chunk<E> load_chunk(const E* row, int e, int H) {
  Chunk<E> c;
#pragma unroll
  for (int i = 0; i < 4 * Chunk<E>::kQ; ++i) c.w[i] = 0;
  if (kVec) {
    if (e < H)
#pragma unroll
      for (int i = 0; i < Chunk<E>::kQ; ++i) c.set(i, load16(reinterpret_cast<const char*>(row + e) + 16 * i));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i < H) c.put(i, row[e + i]);
  }
  return c;
}
template <typename E>
__device__ __forceinline__ Eight pairs(const Chunk<E>& c) {
  Eight v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p[i] = c.pair(i);
  return v;
}
template <typename E, bool kVec>
__device__ __forceinline__ void store_chunk(E* row, int e, int H, const Eight& v) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2(v.p[i]);
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
  if (kVec) {
    if (e < H) store8(row + e, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i < H) store_one(row + e + i, f[i]);
  }
}
// A float32 parameter (a gate row), likewise.
template <bool kVec>
__device__ __forceinline__ Eight load_param(const float* row, int e, int H) {
  return pairs(load_chunk<float, kVec>(row, e, H));
}
// 8 floats of shared memory (the weights, zero-padded to whole chunks).
__device__ __forceinline__ Eight shared8(const float* p) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p), b = *reinterpret_cast<const ulonglong2*>(p + 4);
  return {{a.x, a.y, b.x, b.y}};
}
__device__ __forceinline__ float pair_sum(F2 p) {
  const float2 f = unpack2(p);
  return f.x + f.y;
}

// The value as the type stores it.
__device__ __forceinline__ F2 round_pair(F2 v, const __nv_bfloat16*) {
  const float2 f = unpack2(v);
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&h);
  return pack2(Packed<__nv_bfloat16>::low(w), Packed<__nv_bfloat16>::high(w));
}
__device__ __forceinline__ F2 round_pair(F2 v, const __half*) {
  const float2 f = unpack2(v);
  const __half2 h = __floats2half2_rn(f.x, f.y);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&h);
  return pack2(Packed<__half>::low(w), Packed<__half>::high(w));
}
__device__ __forceinline__ F2 round_pair(F2 v, const float*) { return v; }

// Sum over the group's threads, the same bits in each.  red: two floats a warp of the CTA,
// used in turn, so one barrier a sum is enough.
struct GroupSum {
  float* red;
  int threads, group, turn;
  __device__ float operator()(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (threads == 32) return x;
    const int warps = threads >> 5, warp = threadIdx.x >> 5;
    float* r = red + turn * 16;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) r[warp] = x;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
    const int w0 = group * warps;
    float s = r[w0];
    for (int w = 1; w < warps; ++w) s += r[w0 + w];
    return s;
  }
};

struct NormArgs {
  const void *x, *y;
  int64_t ldx, ldy, T;
  int H, group;
  const float *weight, *gate, *next_weight;
  int64_t rows_per_gate;   // 0: gate is one number a row
  float alpha, eps;
  void *r, *n;
  float *rstd_y, *rstd_r;
};

// The weights in shared memory, padded with zeros to the threads' chunks.
__device__ __forceinline__ void stage_weight(float* dst, const float* w, int H, int padded) {
  for (int i = threadIdx.x; i < padded; i += blockDim.x) dst[i] = w != nullptr && i < H ? w[i] : 0.f;
}

// kBranch: r = alpha x + gate norm(y); else r is x itself and is not written.
// The weights live in shared memory, so that a thread needs few registers and enough rows are
// in flight: 1024 threads an SM hold 64 bytes each of the rows they wait for.
template <typename E, bool kBranch, bool kNext, bool kVec>
__global__ void __launch_bounds__(512, 2) block_norm_kernel(const NormArgs a) {
  extern __shared__ __align__(16) float weights[];
  __shared__ float red[32];
  const int G = a.group, groups = blockDim.x / G, group = threadIdx.x / G, tid = threadIdx.x % G;
  const int padded = 8 * kChunks * G;
  float *w = weights, *wn = weights + (kBranch ? padded : 0);
  if (kBranch) stage_weight(w, a.weight, a.H, padded);
  if (kNext) stage_weight(wn, a.next_weight, a.H, padded);
  __syncthreads();
  GroupSum sum{red, G, group, 0};
  const float inv_h = 1.f / a.H;
  const bool per_token = a.gate != nullptr && a.rows_per_gate == 0;
  const F2 alpha = pack2(a.alpha, a.alpha);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * groups + group; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * groups) {
    Chunk<E> xr[kChunks], yr[kChunks];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int e = 8 * (tid + j * G);
      if (kBranch) yr[j] = load_chunk<E, kVec>(static_cast<const E*>(a.y) + t * a.ldy, e, a.H);
      xr[j] = load_chunk<E, kVec>(static_cast<const E*>(a.x) + t * a.ldx, e, a.H);
    }
    Eight x[kChunks];
    if (kBranch) {
      F2 ss = 0;
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(yr[j].pair(i), yr[j].pair(i), ss);
      const float rstd = rsqrtf(fmaf(sum(pair_sum(ss)), inv_h, a.eps));
      if (tid == 0) a.rstd_y[t] = rstd;
      const float f = per_token ? rstd * a.gate[t] : rstd;
      const F2 ff = pack2(f, f);
      const float* grow = a.gate != nullptr && !per_token ? a.gate + t / a.rows_per_gate * a.H : nullptr;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const int e = 8 * (tid + j * G);
        const Eight wj = shared8(w + e);
        Eight y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y.p[i] = mul2(mul2(yr[j].pair(i), ff), wj.p[i]);
        if (grow != nullptr) {
          const Eight g = load_param<kVec>(grow, e, a.H);
#pragma unroll
          for (int i = 0; i < 4; ++i) y.p[i] = mul2(y.p[i], g.p[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[j].p[i] = round_pair(fma2(alpha, xr[j].pair(i), y.p[i]), static_cast<const E*>(nullptr));
        store_chunk<E, kVec>(static_cast<E*>(a.r) + t * a.H, e, a.H, x[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kChunks; ++j) x[j] = pairs(xr[j]);
    }
    if (kNext) {
      F2 ss = 0;
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(x[j].p[i], x[j].p[i], ss);
      const float rstd = rsqrtf(fmaf(sum(pair_sum(ss)), inv_h, a.eps));
      if (tid == 0) a.rstd_r[t] = rstd;
      const F2 rr = pack2(rstd, rstd);
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const int e = 8 * (tid + j * G);
        const Eight wj = shared8(wn + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[j].p[i] = mul2(mul2(x[j].p[i], rr), wj.p[i]);
        store_chunk<E, kVec>(static_cast<E*>(a.n) + t * a.H, e, a.H, x[j]);
      }
    }
  }
}

struct NormBackwardArgs {
  const void *dr, *dn, *r, *y;   // dr nullable
  int64_t lddr, lddn, ldr, ldy, T;
  int H, group;
  const float *rstd_y, *rstd_r, *weight, *gate, *next_weight;
  int64_t rows_per_gate;
  float alpha;
  void *dx, *dy;
  float* dgate_token;            // one number a row (per-token gates)
  float *part_w, *part_n;        // [parts, H]: sums over a range of rows
  int64_t segment, parts;        // rows that share a gate row; ranges a segment
};

// With d the gradient at r:
//   d = dr + rstd_r (dn w' - rhat mean(dn w' rhat)),  rhat = r rstd_r      (kNext)
//   dx = alpha d;  v = d gate w;  dy = rstd_y (v - yhat mean(v yhat))       (kBranch)
//   sums over rows: d yhat (per-token: times the gate), dn rhat
template <typename E, bool kBranch, bool kNext, bool kVec>
__global__ void __launch_bounds__(512) block_norm_backward_kernel(const NormBackwardArgs a) {
  extern __shared__ __align__(16) float weights[];   // w, w'; at the end the groups' column sums
  __shared__ float red[32];
  const int G = a.group, groups = blockDim.x / G, group = threadIdx.x / G, tid = threadIdx.x % G;
  const int padded = 8 * kChunks * G;
  float *w = weights, *wn = weights + (kBranch ? padded : 0);
  if (kBranch) stage_weight(w, a.weight, a.H, padded);
  if (kNext) stage_weight(wn, a.next_weight, a.H, padded);
  __syncthreads();
  GroupSum sum{red, G, group, 0};
  const int64_t seg = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const int64_t per = (a.segment + a.parts - 1) / a.parts;
  const int64_t row0 = seg * a.segment + part * per;
  const int64_t row1 = seg * a.segment + (part * per + per < a.segment ? part * per + per : a.segment);
  const bool per_token = a.gate != nullptr && a.rows_per_gate == 0;
  const float* grow = a.gate != nullptr && !per_token ? a.gate + seg * a.H : nullptr;
  Eight acc_w[kChunks], acc_n[kChunks];
#pragma unroll
  for (int j = 0; j < kChunks; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc_w[j].p[i] = acc_n[j].p[i] = 0;
  const float inv_h = 1.f / a.H;
  const F2 alpha = pack2(a.alpha, a.alpha);
  for (int64_t t = row0 + group; t < row1; t += groups) {
    Chunk<E> dr[kChunks], dnr[kChunks], rr[kChunks], yr[kChunks];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int e = 8 * (tid + j * G);
      if (kNext) {
        dnr[j] = load_chunk<E, kVec>(static_cast<const E*>(a.dn) + t * a.lddn, e, a.H);
        rr[j] = load_chunk<E, kVec>(static_cast<const E*>(a.r) + t * a.ldr, e, a.H);
      }
      dr[j] = load_chunk<E, kVec>(static_cast<const E*>(a.dr) + t * a.lddr, e, a.dr != nullptr ? a.H : 0);
      if (kBranch) yr[j] = load_chunk<E, kVec>(static_cast<const E*>(a.y) + t * a.ldy, e, a.H);
    }
    Eight d[kChunks];
    if (kNext) {
      const float rstd = a.rstd_r[t];
      const F2 rs = pack2(rstd, rstd);
      F2 dot = 0;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const Eight wj = shared8(wn + 8 * (tid + j * G));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 rhat = mul2(rr[j].pair(i), rs), dn = dnr[j].pair(i);
          acc_n[j].p[i] = fma2(dn, rhat, acc_n[j].p[i]);
          d[j].p[i] = mul2(dn, wj.p[i]);
          dot = fma2(d[j].p[i], rhat, dot);
        }
      }
      const float m = -sum(pair_sum(dot)) * inv_h * rstd;   // times r, not rhat, below
      const F2 mm = pack2(m, m);
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          d[j].p[i] = fma2(rs, fma2(mm, rr[j].pair(i), d[j].p[i]), dr[j].pair(i));
    } else {
#pragma unroll
      for (int j = 0; j < kChunks; ++j) d[j] = pairs(dr[j]);
    }
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      Eight v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v.p[i] = mul2(alpha, d[j].p[i]);
      store_chunk<E, kVec>(static_cast<E*>(a.dx) + t * a.H, 8 * (tid + j * G), a.H, v);
    }
    if (kBranch) {
      const float rstd = a.rstd_y[t];
      const float gt = per_token ? a.gate[t] : 1.f;
      const F2 rs = pack2(rstd, rstd), gg = pack2(gt, gt);
      F2 dot = 0;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const int e = 8 * (tid + j * G);
        const Eight wj = shared8(w + e);
        Eight g;
        if (grow != nullptr) g = load_param<kVec>(grow, e, a.H);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 yhat = mul2(yr[j].pair(i), rs);
          acc_w[j].p[i] = fma2(mul2(gg, d[j].p[i]), yhat, acc_w[j].p[i]);
          d[j].p[i] = mul2(d[j].p[i], wj.p[i]);
          if (grow != nullptr) d[j].p[i] = mul2(d[j].p[i], g.p[i]);
          dot = fma2(d[j].p[i], yhat, dot);
        }
      }
      const float s = sum(pair_sum(dot));   // the token gate's gradient; the mean below times the gate
      if (per_token && tid == 0) a.dgate_token[t] = s;
      const float m = -s * inv_h * rstd, f = rstd * gt;
      const F2 mm = pack2(m, m), ff = pack2(f, f);
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[j].p[i] = mul2(ff, fma2(mm, yr[j].pair(i), d[j].p[i]));
        store_chunk<E, kVec>(static_cast<E*>(a.dy) + t * a.H, 8 * (tid + j * G), a.H, d[j]);
      }
    }
  }
  // the groups' column sums, added in order, one row of the parts a CTA
  for (int which = 0; which < 2; ++which) {
    if (which == 0 ? !kBranch : !kNext) continue;
    float* out = (which == 0 ? a.part_w : a.part_n) + static_cast<int64_t>(blockIdx.x) * a.H;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<F2*>(weights + group * padded + 8 * (tid + j * G) + 2 * i) =
            which == 0 ? acc_w[j].p[i] : acc_n[j].p[i];
    __syncthreads();
    for (int e = threadIdx.x; e < a.H; e += blockDim.x) {
      float s = weights[e];
      for (int g = 1; g < groups; ++g) s += weights[g * padded + e];
      out[e] = s;
    }
  }
}

struct NormReduceArgs {
  const float *part_w, *part_n, *weight, *gate;   // gate: rows of H, or null
  int H;
  int64_t segments, parts;
  float *dweight, *dgate, *dnext;                 // nullable
};

constexpr int kReduceSlices = 16;

// CTA (b, s): 32 columns, a warp a slice of the ranges.  s = 0, 1: the two weights' gradients over all
// ranges; s > 1: the gradient of gate row s - 2.
__global__ void __launch_bounds__(32 * kReduceSlices) block_norm_reduce_kernel(const NormReduceArgs a) {
  __shared__ float red[kReduceSlices][32];
  const int blocks = (a.H + 31) / 32, lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int e = static_cast<int>(blockIdx.x % blocks) * 32 + lane;
  const int64_t s = blockIdx.x / blocks;
  float* out = s == 0 ? a.dweight : s == 1 ? a.dnext : a.dgate + (s - 2) * a.H;
  if (out == nullptr) return;
  const float* src = s == 1 ? a.part_n : a.part_w;
  const int64_t first = s < 2 ? 0 : (s - 2) * a.parts, count = s < 2 ? a.segments * a.parts : a.parts;
  const bool gated = s == 0 && a.gate != nullptr;
  float v = 0.f;
  if (e < a.H) {
#pragma unroll 8
    for (int64_t p = slice; p < count; p += kReduceSlices) {
      const float x = src[(first + p) * a.H + e];
      v = gated ? fmaf(a.gate[p / a.parts * a.H + e], x, v) : v + x;
    }
  }
  red[slice][lane] = v;
  __syncthreads();
  if (slice == 0 && e < a.H) {
#pragma unroll
    for (int i = 1; i < kReduceSlices; ++i) v += red[i][lane];
    out[e] = s > 1 ? v * a.weight[e] : v;
  }
}

bool rows_aligned(const void* p, int64_t ld, int e) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * e % 16 == 0);
}

// Launches with more than 48 KB of shared memory (H > 4096: two weights of 32 KB) need the limit raised.
template <typename Args>
cudaError_t start(void (*kernel)(Args), dim3 grid, int threads, size_t smem, cudaStream_t s, const Args& a) {
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, threads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename E>
cudaError_t forward(const NormArgs& a, cudaStream_t s) {
  const int e = sizeof(E);
  const bool vec = a.H % 8 == 0 && rows_aligned(a.x, a.ldx, e) && rows_aligned(a.y, a.ldy, e) &&
                   rows_aligned(a.r, a.H, e) && rows_aligned(a.n, a.H, e) && rows_aligned(a.weight, a.H, 4) &&
                   rows_aligned(a.next_weight, a.H, 4) &&
                   (a.rows_per_gate == 0 || rows_aligned(a.gate, a.H, 4));
  const int threads = a.group > kNormThreads ? a.group : kNormThreads, groups = threads / a.group;
  const int64_t want = (a.T + groups - 1) / groups, most = static_cast<int64_t>(num_sms()) * (1024 / threads);
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  const bool branch = a.y != nullptr, next = a.next_weight != nullptr;
  const size_t smem = sizeof(float) * 8 * kChunks * a.group * ((branch ? 1 : 0) + (next ? 1 : 0));   // at most 64 KB
#define NVFP4_NORM(B, N, V) return start(block_norm_kernel<E, B, N, V>, grid, threads, smem, s, a)
  if (vec) {
    if (branch && next) NVFP4_NORM(true, true, true);
    else if (branch) NVFP4_NORM(true, false, true);
    else NVFP4_NORM(false, true, true);
  } else {
    if (branch && next) NVFP4_NORM(true, true, false);
    else if (branch) NVFP4_NORM(true, false, false);
    else NVFP4_NORM(false, true, false);
  }
#undef NVFP4_NORM
}

template <typename E>
cudaError_t backward(const NormBackwardArgs& a, int64_t segments, float* dweight, float* dgate, float* dnext,
                     cudaStream_t s) {
  const int e = sizeof(E);
  const bool vec = a.H % 8 == 0 && rows_aligned(a.dr, a.lddr, e) && rows_aligned(a.dn, a.lddn, e) &&
                   rows_aligned(a.r, a.ldr, e) && rows_aligned(a.y, a.ldy, e) && rows_aligned(a.dx, a.H, e) &&
                   rows_aligned(a.dy, a.H, e) && rows_aligned(a.weight, a.H, 4) &&
                   rows_aligned(a.next_weight, a.H, 4) && (a.rows_per_gate == 0 || rows_aligned(a.gate, a.H, 4));
  const int threads = a.group > kNormThreads ? a.group : kNormThreads, groups = threads / a.group;
  const dim3 grid(static_cast<unsigned>(segments * a.parts));
  const bool branch = a.y != nullptr, next = a.next_weight != nullptr;
  const int rows = (branch ? 1 : 0) + (next ? 1 : 0);   // of shared memory: the weights, later the groups' sums
  const size_t smem = sizeof(float) * 8 * kChunks * a.group * (rows > groups ? rows : groups);
  cudaError_t err;
#define NVFP4_NORM(B, N, V) err = start(block_norm_backward_kernel<E, B, N, V>, grid, threads, smem, s, a)
  if (vec) {
    if (branch && next) NVFP4_NORM(true, true, true);
    else if (branch) NVFP4_NORM(true, false, true);
    else NVFP4_NORM(false, true, true);
  } else {
    if (branch && next) NVFP4_NORM(true, true, false);
    else if (branch) NVFP4_NORM(true, false, false);
    else NVFP4_NORM(false, true, false);
  }
#undef NVFP4_NORM
  if (err != cudaSuccess) return err;
  NormReduceArgs ra{a.part_w, a.part_n, a.weight, a.rows_per_gate > 0 ? a.gate : nullptr, a.H, segments, a.parts,
                    dweight, a.rows_per_gate > 0 ? dgate : nullptr, dnext};
  const int64_t blocks = (a.H + 31) / 32;
  block_norm_reduce_kernel<<<static_cast<unsigned>(blocks * (2 + (ra.gate != nullptr ? segments : 0))),
                             32 * kReduceSlices, 0, s>>>(ra);
  return cudaGetLastError();
}

constexpr int64_t kNormParts = 304;   // ranges of rows in all, unless there are more gate rows

}  // namespace

int64_t block_norm_parts(int64_t T, int64_t gate_rows) {
  const int64_t segments = gate_rows > 0 ? gate_rows : 1, rows = T / segments;
  int64_t parts = kNormParts / segments;
  if (parts > rows) parts = rows;
  return parts > 0 ? parts : 1;
}

cudaError_t launch_block_norm(const void* x, int64_t ldx, const void* y, int64_t ldy, int dtype, int64_t T, int64_t H,
                              const float* weight, const float* gate, int64_t gate_rows, float alpha,
                              const float* next_weight, float eps, void* r, void* n, float* rstd_y, float* rstd_r,
                              cudaStream_t s) {
  NormArgs a{x, y, ldx, ldy, T, static_cast<int>(H), group_threads(H), weight, gate, next_weight,
             gate_rows > 0 ? T / gate_rows : 0, alpha, eps, r, n, rstd_y, rstd_r};
  if (dtype == kActBF16) return forward<__nv_bfloat16>(a, s);
  if (dtype == kActF16) return forward<__half>(a, s);
  return forward<float>(a, s);
}

cudaError_t launch_block_norm_backward(const void* dr, int64_t lddr, const void* dn, int64_t lddn, const void* r,
                                       int64_t ldr, const void* y, int64_t ldy, int dtype, int64_t T, int64_t H,
                                       const float* rstd_y, const float* rstd_r, const float* weight,
                                       const float* gate, int64_t gate_rows, float alpha, const float* next_weight,
                                       void* dx, void* dy, float* dweight, float* dgate, float* dnext, float* partial,
                                       cudaStream_t s) {
  const int64_t segments = gate_rows > 0 ? gate_rows : 1, parts = block_norm_parts(T, gate_rows);
  NormBackwardArgs a{dr,     dn,    r,    y,    lddr,        lddn,
                     ldr,    ldy,   T,    static_cast<int>(H), group_threads(H), rstd_y,
                     rstd_r, weight, gate, next_weight, gate_rows > 0 ? T / gate_rows : 0, alpha,
                     dx,     dy,    gate_rows > 0 ? nullptr : dgate, partial, partial + segments * parts * H,
                     T / segments, parts};
  if (dtype == kActBF16) return backward<__nv_bfloat16>(a, segments, dweight, dgate, dnext, s);
  if (dtype == kActF16) return backward<__half>(a, segments, dweight, dgate, dnext, s);
  return backward<float>(a, segments, dweight, dgate, dnext, s);
}

}  // namespace nvfp4
