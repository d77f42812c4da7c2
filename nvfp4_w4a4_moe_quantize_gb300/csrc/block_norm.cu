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

template <typename E, bool kVec>
struct RowIo {
  // chunk j of this thread: elements [e, e + 8)
  static __device__ __forceinline__ void load(const E* row, int e, int H, float (&v)[8]) {
    if (kVec) {
      if (e < H) {
        Chunk<E> c;
#pragma unroll
        for (int i = 0; i < Chunk<E>::kQ; ++i) c.q[i] = load16(reinterpret_cast<const char*>(row + e) + 16 * i);
        unpack8(c, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = e + i < H ? to_f32(row[e + i]) : 0.f;
    }
  }
  static __device__ __forceinline__ void store(E* row, int e, int H, const float (&v)[8]) {
    if (kVec) {
      if (e < H) store8(row + e, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e + i < H) store_one(row + e + i, v[i]);
    }
  }
};
// float32 parameters (weights, gates): 16-byte aligned rows or element by element
template <bool kVec>
__device__ __forceinline__ void load_param(const float* row, int e, int H, float (&v)[8]) {
  if (kVec) {
    if (e < H) {
      const float4 a = *reinterpret_cast<const float4*>(row + e), b = *reinterpret_cast<const float4*>(row + e + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = e + i < H ? row[e + i] : 0.f;
  }
}

__device__ __forceinline__ float round_to(float v, const __nv_bfloat16*) { return to_f32(__float2bfloat16_rn(v)); }
__device__ __forceinline__ float round_to(float v, const __half*) { return to_f32(__float2half_rn(v)); }
__device__ __forceinline__ float round_to(float v, const float*) { return v; }

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

// kBranch: r = alpha x + gate norm(y); else r is x itself and is not written.
template <typename E, bool kBranch, bool kNext, bool kVec>
__global__ void __launch_bounds__(512) block_norm_kernel(const NormArgs a) {
  __shared__ float red[32];
  const int G = a.group, groups = blockDim.x / G, group = threadIdx.x / G, tid = threadIdx.x % G;
  GroupSum sum{red, G, group, 0};
  using Io = RowIo<E, kVec>;
  float w[kChunks][8], wn[kChunks][8];
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int e = 8 * (tid + j * G);
    if (kBranch) load_param<kVec>(a.weight, e, a.H, w[j]);
    if (kNext) load_param<kVec>(a.next_weight, e, a.H, wn[j]);
  }
  const float inv_h = 1.f / a.H;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * groups + group; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * groups) {
    float x[kChunks][8], y[kChunks][8];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int e = 8 * (tid + j * G);
      if (kBranch) Io::load(static_cast<const E*>(a.y) + t * a.ldy, e, a.H, y[j]);
      Io::load(static_cast<const E*>(a.x) + t * a.ldx, e, a.H, x[j]);
    }
    if (kBranch) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(y[j][i], y[j][i], ss);
      const float rstd = rsqrtf(fmaf(sum(ss), inv_h, a.eps));
      if (tid == 0) a.rstd_y[t] = rstd;
      const bool per_token = a.gate != nullptr && a.rows_per_gate == 0;
      const float f = per_token ? rstd * a.gate[t] : rstd;
      const float* grow = a.gate != nullptr && !per_token ? a.gate + t / a.rows_per_gate * a.H : nullptr;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const int e = 8 * (tid + j * G);
        float g[8];
        if (grow != nullptr) load_param<kVec>(grow, e, a.H, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float b = y[j][i] * f * w[j][i];
          if (grow != nullptr) b *= g[i];
          x[j][i] = round_to(fmaf(a.alpha, x[j][i], b), static_cast<const E*>(nullptr));
        }
        Io::store(static_cast<E*>(a.r) + t * a.H, e, a.H, x[j]);
      }
    }
    if (kNext) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[j][i], x[j][i], ss);
      const float rstd = rsqrtf(fmaf(sum(ss), inv_h, a.eps));
      if (tid == 0) a.rstd_r[t] = rstd;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const int e = 8 * (tid + j * G);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] = x[j][i] * rstd * wn[j][i];
        Io::store(static_cast<E*>(a.n) + t * a.H, e, a.H, x[j]);
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
  extern __shared__ float cols[];
  __shared__ float red[32];
  const int G = a.group, groups = blockDim.x / G, group = threadIdx.x / G, tid = threadIdx.x % G;
  GroupSum sum{red, G, group, 0};
  using Io = RowIo<E, kVec>;
  const int64_t seg = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const int64_t per = (a.segment + a.parts - 1) / a.parts;
  const int64_t row0 = seg * a.segment + part * per;
  const int64_t row1 = seg * a.segment + (part * per + per < a.segment ? part * per + per : a.segment);
  const bool per_token = a.gate != nullptr && a.rows_per_gate == 0;
  const float* grow = a.gate != nullptr && !per_token ? a.gate + seg * a.H : nullptr;
  float acc_w[kChunks][8], acc_n[kChunks][8];
#pragma unroll
  for (int j = 0; j < kChunks; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc_w[j][i] = acc_n[j][i] = 0.f;
  const float inv_h = 1.f / a.H;
  for (int64_t t = row0 + group; t < row1; t += groups) {
    float d[kChunks][8], dn[kChunks][8], r[kChunks][8], y[kChunks][8];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int e = 8 * (tid + j * G);
      if (kNext) {
        Io::load(static_cast<const E*>(a.dn) + t * a.lddn, e, a.H, dn[j]);
        Io::load(static_cast<const E*>(a.r) + t * a.ldr, e, a.H, r[j]);
      }
      if (a.dr != nullptr) {
        Io::load(static_cast<const E*>(a.dr) + t * a.lddr, e, a.H, d[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[j][i] = 0.f;
      }
      if (kBranch) Io::load(static_cast<const E*>(a.y) + t * a.ldy, e, a.H, y[j]);
    }
    if (kNext) {
      const float rstd = a.rstd_r[t];
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        float wn[8];
        load_param<kVec>(a.next_weight, 8 * (tid + j * G), a.H, wn);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          r[j][i] *= rstd;
          acc_n[j][i] = fmaf(dn[j][i], r[j][i], acc_n[j][i]);
          dn[j][i] *= wn[i];
          dot = fmaf(dn[j][i], r[j][i], dot);
        }
      }
      const float m = sum(dot) * inv_h;
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) d[j][i] = fmaf(rstd, fmaf(-m, r[j][i], dn[j][i]), d[j][i]);
    }
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = a.alpha * d[j][i];
      Io::store(static_cast<E*>(a.dx) + t * a.H, 8 * (tid + j * G), a.H, v);
    }
    if (kBranch) {
      const float rstd = a.rstd_y[t];
      const float gt = per_token ? a.gate[t] : 1.f;
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const int e = 8 * (tid + j * G);
        float w[8], g[8];
        load_param<kVec>(a.weight, e, a.H, w);
        if (grow != nullptr) load_param<kVec>(grow, e, a.H, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[j][i] *= rstd;
          acc_w[j][i] = fmaf(gt * d[j][i], y[j][i], acc_w[j][i]);
          d[j][i] *= w[i];
          if (grow != nullptr) d[j][i] *= g[i];
          dot = fmaf(d[j][i], y[j][i], dot);
        }
      }
      const float s = sum(dot);   // the token gate's gradient; the mean below times the gate
      if (per_token && tid == 0) a.dgate_token[t] = s;
      const float m = s * inv_h, f = rstd * gt;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[j][i] = f * fmaf(-m, y[j][i], d[j][i]);
        Io::store(static_cast<E*>(a.dy) + t * a.H, 8 * (tid + j * G), a.H, d[j]);
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
      for (int i = 0; i < 8; ++i) {
        const int e = 8 * (tid + j * G) + i;
        if (e < a.H) cols[group * a.H + e] = which == 0 ? acc_w[j][i] : acc_n[j][i];
      }
    __syncthreads();
    for (int e = threadIdx.x; e < a.H; e += blockDim.x) {
      float s = cols[e];
      for (int g = 1; g < groups; ++g) s += cols[g * a.H + e];
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

// CTA (b, s): 32 columns, by 8 threads each.  s = 0: the weights' gradients over all ranges;
// s > 0: the gradient of gate row s - 1.
__global__ void __launch_bounds__(256) block_norm_reduce_kernel(const NormReduceArgs a) {
  __shared__ float red[8][33];
  const int blocks = (a.H + 31) / 32, lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int e = static_cast<int>(blockIdx.x % blocks) * 32 + lane;
  const int64_t s = blockIdx.x / blocks;
  const int64_t first = s == 0 ? 0 : (s - 1) * a.parts, count = s == 0 ? a.segments * a.parts : a.parts;
  for (int which = 0; which < 2; ++which) {
    float* out = which == 1 ? a.dnext : (s == 0 ? a.dweight : a.dgate + (s - 1) * a.H);
    if ((which == 1 && s > 0) || out == nullptr) continue;
    const float* src = which == 0 ? a.part_w : a.part_n;
    float v = 0.f;
    if (e < a.H)
      for (int64_t p = slice; p < count; p += 8) {
        const float x = src[(first + p) * a.H + e];
        v = which == 0 && s == 0 && a.gate != nullptr ? fmaf(a.gate[p / a.parts * a.H + e], x, v) : v + x;
      }
    red[slice][lane] = v;
    __syncthreads();
    if (slice == 0 && e < a.H) {
      for (int i = 1; i < 8; ++i) v += red[i][lane];
      out[e] = which == 0 && s > 0 ? v * a.weight[e] : v;
    }
    __syncthreads();
  }
}

bool rows_aligned(const void* p, int64_t ld, int e) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * e % 16 == 0);
}

template <typename E>
cudaError_t forward(const NormArgs& a, cudaStream_t s) {
  const int e = sizeof(E);
  const bool vec = a.H % 8 == 0 && rows_aligned(a.x, a.ldx, e) && rows_aligned(a.y, a.ldy, e) &&
                   rows_aligned(a.r, a.H, e) && rows_aligned(a.n, a.H, e) && rows_aligned(a.weight, a.H, 4) &&
                   rows_aligned(a.next_weight, a.H, 4) &&
                   (a.rows_per_gate == 0 || rows_aligned(a.gate, a.H, 4));
  const int threads = a.group > kNormThreads ? a.group : kNormThreads, groups = threads / a.group;
  const int64_t want = (a.T + groups - 1) / groups, most = static_cast<int64_t>(num_sms()) * 8;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  const bool branch = a.y != nullptr, next = a.next_weight != nullptr;
#define NVFP4_NORM(B, N, V) block_norm_kernel<E, B, N, V><<<grid, threads, 0, s>>>(a)
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
  return cudaGetLastError();
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
  const size_t smem = sizeof(float) * groups * a.H;   // at most 256 / G * 16 G floats: 16 KB, 32 KB for G = 512
  const bool branch = a.y != nullptr, next = a.next_weight != nullptr;
#define NVFP4_NORM(B, N, V) block_norm_backward_kernel<E, B, N, V><<<grid, threads, smem, s>>>(a)
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
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  NormReduceArgs ra{a.part_w, a.part_n, a.weight, a.rows_per_gate > 0 ? a.gate : nullptr, a.H, segments, a.parts,
                    dweight, a.rows_per_gate > 0 ? dgate : nullptr, dnext};
  const int64_t blocks = (a.H + 31) / 32;
  block_norm_reduce_kernel<<<static_cast<unsigned>(blocks * (1 + (ra.gate != nullptr ? segments : 0))), 256, 0, s>>>(ra);
  return cudaGetLastError();
}

constexpr int64_t kNormParts = 608;   // ranges of rows in all, unless there are more gate rows

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
