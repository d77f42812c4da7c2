// RMS norms before and after the expert block, fused with the block's gate and the residual's
// scale, and their backward.
//
//   n = x rstd(x) w                                    rstd(x) = 1 / sqrt(mean(x^2) + eps)
//   r = a x + gate (y rstd(y) w);   n' = r rstd(r) w'  (r as it is stored)
//
// A row stays on the SM between its reductions: x and y are read once, r and n' written
// once.  A row belongs to a group of G threads, G a function of H alone, 16 elements a
// thread; sums run in an order that H fixes, so a row's bits do not depend on the batch.
// What bounds these kernels is HBM, if enough bytes are on their way: a group's next rows arrive in
// shared memory by bulk copies while it works on one, and the weights stay there.  If one of
// the arrays has rows that are not 16-byte aligned, all are read and written element by
// element, with no row ahead, and the backward spills registers; where the width is a multiple of 8 all
// the same, a thread's elements are neighbours and a warp's reads do not coalesce.
// Backward: a CTA takes a range of rows of one gate row and keeps the column sums of the
// weights' and gate's gradients in registers; the ranges' sums are added by a second kernel
// in a fixed order (no atomics).
// Measured at 32768 x 2048 BF16 with a gate a token and the next norm: forward 90 us (6.0 TB/s, 88% of
// a copy's rate), backward 139 us (5.8 TB/s) of which the second kernel takes 5; the norm before the block 53 us
// (5.0 TB/s), backward 103 us (5.2 TB/s).  Not aligned, forward and backward: 213 and 566 us at a width of
// 2047, 400 and 615 us at a width of 2048 and a pitch of 2051.  Both use 50-60% of the issue
// slots; more rows ahead, other numbers of CTAs, and 8 or 32 elements a thread were slower
// (forward 91-123 us, backward 142-198 us).
#include "launch.h"
#include "pdl.cuh"
#include "ptx.cuh"
#include "status.cuh"
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

// 8 values as pairs.
struct Eight {
  F2 p[4];
};

// The elements of a thread's chunk: first, first + step, ... (8 of them, below H).  Where H is a
// multiple of 8 they are neighbours, else a group apart, so that single reads coalesce.
struct Places {
  int first, step, H;
};
template <bool kVec>   // rows are 16-byte aligned and whole chunks of neighbours
__device__ __forceinline__ Places places(int tid, int j, int G, int H) {
  return kVec || H % 8 == 0 ? Places{8 * (tid + j * G), 1, H} : Places{tid + 8 * j * G, G, H};
}

template <typename E, bool kVec>
__device__ __forceinline__ Chunk<E> load_chunk(const E* row, const Places& at) {
  Chunk<E> c;
#pragma unroll
  for (int i = 0; i < 4 * Chunk<E>::kQ; ++i) c.w[i] = 0;
  if (kVec) {
    if (at.first < at.H)
#pragma unroll
      for (int i = 0; i < Chunk<E>::kQ; ++i) c.set(i, load16(reinterpret_cast<const char*>(row + at.first) + 16 * i));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at.first + i * at.step < at.H) c.put(i, row[at.first + i * at.step]);
  }
  return c;
}
template <typename E>
__device__ __forceinline__ Chunk<E> stage_chunk(const char* row, const Places& at) {
  Chunk<E> c;
#pragma unroll
  for (int i = 0; i < 4 * Chunk<E>::kQ; ++i) c.w[i] = 0;
  if (at.first < at.H)
#pragma unroll
    for (int i = 0; i < Chunk<E>::kQ; ++i)
      c.set(i, reinterpret_cast<const uint4*>(row + at.first * sizeof(E))[i]);
  return c;
}
template <typename E>
__device__ __forceinline__ Eight pairs(const Chunk<E>& c) {
  Eight v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p[i] = c.pair(i);
  return v;
}
// A float32 parameter (a gate row), likewise.
template <bool kVec>
__device__ __forceinline__ Eight load_param(const float* row, const Places& at) {
  return pairs(load_chunk<float, kVec>(row, at));
}
// The weights, in shared memory and zero beyond H.
template <bool kVec>
__device__ __forceinline__ Eight shared8(const float* w, const Places& at) {
  Eight v;
  if (kVec) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(w + at.first);
    const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(w + at.first + 4);
    v.p[0] = a.x;
    v.p[1] = a.y;
    v.p[2] = b.x;
    v.p[3] = b.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v.p[i] = pack2(w[at.first + 2 * i * at.step], w[at.first + (2 * i + 1) * at.step]);
  }
  return v;
}
__device__ __forceinline__ float pair_sum(F2 p) {
  const float2 f = unpack2(p);
  return f.x + f.y;
}

// Pairs as the type stores them.
template <typename E>
__device__ __forceinline__ Chunk<E> stored(const Eight& v) {
  Chunk<E> c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(v.p[i]);
    if constexpr (sizeof(E) == 4) {
      c.w[2 * i] = __float_as_uint(f.x);
      c.w[2 * i + 1] = __float_as_uint(f.y);
    } else if constexpr (std::is_same_v<E, __half>) {
      const __half2 h = __floats2half2_rn(f.x, f.y);
      c.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
      c.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return c;
}
template <typename E, bool kVec>
__device__ __forceinline__ void store_chunk(E* row, const Places& at, const Chunk<E>& c) {
  if (kVec) {
    if (at.first < at.H)
#pragma unroll
      for (int i = 0; i < Chunk<E>::kQ; ++i)
        reinterpret_cast<uint4*>(row + at.first)[i] =
            make_uint4(c.w[4 * i], c.w[4 * i + 1], c.w[4 * i + 2], c.w[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (at.first + i * at.step < at.H) row[at.first + i * at.step] = c.get(i);
  }
}
template <typename E, bool kVec>
__device__ __forceinline__ void store_chunk(E* row, const Places& at, const Eight& v) {
  store_chunk<E, kVec>(row, at, stored<E>(v));
}

// Sum over the group's threads, the same bits in each.  red: two floats a warp of the CTA,
// used in turn, so one barrier a sum is enough.
struct GroupSum {
  float* red;
  int threads, group, turn;
  __device__ __forceinline__ void sync() const {
    if (threads > 32) asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory");
  }
  __device__ float operator()(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (threads == 32) return x;
    const int warps = threads >> 5, warp = threadIdx.x >> 5;
    float* r = red + turn * 16;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) r[warp] = x;
    sync();
    const int w0 = group * warps;
    float s = r[w0];
    for (int w = 1; w < warps; ++w) s += r[w0 + w];
    return s;
  }
};

// A group's rows on their way into shared memory: `stages` rows of N arrays each.
constexpr int kMaxStages = 4;
template <int N>
struct Ring {
  char* mem;            // this group's
  uint64_t* bars;
  int stages, row_bytes;
  int at = 0, parity = 0;
  __device__ __forceinline__ char* array(int i) const { return mem + (at * N + i) * row_bytes; }
  // One thread: starts row number k (k = 0, 1, ... of the group) of the arrays that are given.
  __device__ __forceinline__ void start(int stage, const void* const (&rows)[N]) const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += rows[i] != nullptr;
    mbar_arrive_expect_tx(&bars[stage], n * row_bytes);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (rows[i] != nullptr) bulk_load(mem + (stage * N + i) * row_bytes, rows[i], row_bytes, &bars[stage]);
  }
  __device__ __forceinline__ void wait(int* status, int* abort) const { mbar_wait(&bars[at], parity, status, abort); }
  __device__ __forceinline__ void next() {
    if (++at == stages) {
      at = 0;
      parity ^= 1;
    }
  }
};

struct NormArgs {
  const void *x, *y;
  int64_t ldx, ldy, T;
  int H, group, stages;
  const float *weight, *gate, *next_weight;
  int64_t rows_per_gate;   // 0: gate is one number a row
  float alpha, eps;
  void *r, *n;
  float *rstd_y, *rstd_r;
  int* status;
};

// The weights in shared memory, padded with zeros to the threads' chunks.
__device__ __forceinline__ void stage_weight(float* dst, const float* w, int H, int padded) {
  for (int i = threadIdx.x; i < padded; i += blockDim.x) dst[i] = w != nullptr && i < H ? w[i] : 0.f;
}

// kBranch: r = alpha x + gate norm(y); else r is x itself and is not written.
// kVec: the rows come through the ring; else from global memory, element by element.
template <typename E, bool kBranch, bool kNext, bool kVec>
__global__ void __launch_bounds__(512, 2) block_norm_kernel(const NormArgs a) {
  constexpr int N = kBranch ? 2 : 1;
  extern __shared__ __align__(128) float weights[];
  __shared__ float red[32];
  __shared__ uint64_t bars[8 * kMaxStages];
  __shared__ int abort;
  const int G = a.group, groups = blockDim.x / G, group = threadIdx.x / G, tid = threadIdx.x % G;
  const int padded = 8 * kChunks * G;
  float *w = weights, *wn = weights + (kBranch ? padded : 0);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * groups + group;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * groups;
  const auto x_row = [&](int64_t t) { return static_cast<const E*>(a.x) + t * a.ldx; };
  const auto y_row = [&](int64_t t) { return static_cast<const E*>(a.y) + t * a.ldy; };
  const int row_bytes = a.H * static_cast<int>(sizeof(E));
  Ring<N> ring{reinterpret_cast<char*>(weights + padded * ((kBranch ? 1 : 0) + (kNext ? 1 : 0))) +
                   static_cast<int64_t>(group) * a.stages * N * row_bytes,
               bars + group * kMaxStages, a.stages, row_bytes};
  const auto start = [&](int stage, int64_t t) {
    if constexpr (kBranch) ring.start(stage, {y_row(t), x_row(t)});
    else ring.start(stage, {x_row(t)});
  };
  if (kVec) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < 8 * kMaxStages; ++i) mbar_init(&bars[i], 1);
      fence_mbar_init();
      abort = 0;
    }
    __syncthreads();
    if (tid == 0)
      for (int k = 0; k < a.stages && t0 + k * stride < a.T; ++k) start(k, t0 + k * stride);
  }
  if (kBranch) stage_weight(w, a.weight, a.H, padded);
  if (kNext) stage_weight(wn, a.next_weight, a.H, padded);
  __syncthreads();
  GroupSum sum{red, G, group, 0};
  const float inv_h = 1.f / a.H;
  const bool per_token = a.gate != nullptr && a.rows_per_gate == 0;
  const F2 alpha = pack2(a.alpha, a.alpha);
  for (int64_t t = t0; t < a.T; t += stride) {
    Chunk<E> xr[kChunks], yr[kChunks];
    if (kVec) ring.wait(a.status, &abort);
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const Places at = places<kVec>(tid, j, G, a.H);
      if (kBranch) yr[j] = kVec ? stage_chunk<E>(ring.array(0), at) : load_chunk<E, false>(y_row(t), at);
      xr[j] = kVec ? stage_chunk<E>(ring.array(N - 1), at) : load_chunk<E, false>(x_row(t), at);
    }
    // once the group has read a row, its place is free for the one after the next
    const auto refill = [&] {
      if (!kVec) return;
      if (G == 32) __syncwarp();
      if (tid == 0 && t + a.stages * stride < a.T) start(ring.at, t + a.stages * stride);
      ring.next();
    };
    if (kBranch) {
      F2 ss = 0;
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(yr[j].pair(i), yr[j].pair(i), ss);
      const float rstd = rsqrtf(fmaf(sum(pair_sum(ss)), inv_h, a.eps));
      refill();
      if (tid == 0) a.rstd_y[t] = rstd;
      const float f = per_token ? rstd * a.gate[t] : rstd;   // (read earlier, 90 instead of 88 us)
      const F2 ff = pack2(f, f);
      const float* grow = a.gate != nullptr && !per_token ? a.gate + t / a.rows_per_gate * a.H : nullptr;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const Places at = places<kVec>(tid, j, G, a.H);
        const Eight wj = shared8<kVec>(w, at);
        Eight y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y.p[i] = mul2(mul2(yr[j].pair(i), ff), wj.p[i]);
        if (grow != nullptr) {
          const Eight g = load_param<kVec>(grow, at);
#pragma unroll
          for (int i = 0; i < 4; ++i) y.p[i] = mul2(y.p[i], g.p[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) y.p[i] = fma2(alpha, xr[j].pair(i), y.p[i]);
        xr[j] = stored<E>(y);
        store_chunk<E, kVec>(static_cast<E*>(a.r) + t * a.H, at, xr[j]);
      }
    }
    if (kNext) {
      F2 ss = 0;
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(xr[j].pair(i), xr[j].pair(i), ss);
      const float rstd = rsqrtf(fmaf(sum(pair_sum(ss)), inv_h, a.eps));
      if (!kBranch) refill();
      if (tid == 0) a.rstd_r[t] = rstd;
      const F2 rr = pack2(rstd, rstd);
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const Places at = places<kVec>(tid, j, G, a.H);
        const Eight wj = shared8<kVec>(wn, at);
        Eight v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v.p[i] = mul2(mul2(xr[j].pair(i), rr), wj.p[i]);
        store_chunk<E, kVec>(static_cast<E*>(a.n) + t * a.H, at, v);
      }
    }
  }
}

struct NormBackwardArgs {
  const void *dr, *dn, *r, *y;   // dr nullable
  int64_t lddr, lddn, ldr, ldy, T;
  int H, group, stages;
  const float *rstd_y, *rstd_r, *weight, *gate, *next_weight;
  int64_t rows_per_gate;
  float alpha;
  void *dx, *dy;
  float* dgate_token;            // one number a row (per-token gates)
  float *part_w, *part_n;        // [parts, H]: sums over a range of rows
  int64_t segment, parts;        // rows that share a gate row; ranges a segment
  int* status;
};

// With d the gradient at r:
//   d = dr + rstd_r (dn w' - rhat mean(dn w' rhat)),  rhat = r rstd_r      (kNext)
//   dx = alpha d;  v = d gate w;  dy = rstd_y (v - yhat mean(v yhat))       (kBranch)
//   sums over rows: d yhat (per-token: times the gate), dn rhat
template <typename E, bool kBranch, bool kNext, bool kVec>
__global__ void __launch_bounds__(512) block_norm_backward_kernel(const NormBackwardArgs a) {
  constexpr int N = 1 + (kBranch ? 1 : 0) + (kNext ? 2 : 0);
  constexpr int kDr = 0, kY = 1, kDn = kBranch ? 2 : 1, kR = kDn + 1;   // arrays of the ring
  extern __shared__ __align__(128) float weights[];   // w, w'; at the end the groups' column sums
  __shared__ float red[32];
  __shared__ uint64_t bars[8 * kMaxStages];
  __shared__ int abort;
  const int G = a.group, groups = blockDim.x / G, group = threadIdx.x / G, tid = threadIdx.x % G;
  const int padded = 8 * kChunks * G;
  float *w = weights, *wn = weights + (kBranch ? padded : 0);
  const int64_t seg = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const int64_t per = (a.segment + a.parts - 1) / a.parts;
  const int64_t row0 = seg * a.segment + part * per + group;
  const int64_t row1 = seg * a.segment + (part * per + per < a.segment ? part * per + per : a.segment);
  const auto row_of = [&](const void* p, int64_t ld, int64_t t) { return static_cast<const E*>(p) + t * ld; };
  const int row_bytes = a.H * static_cast<int>(sizeof(E));
  Ring<N> ring{reinterpret_cast<char*>(weights + padded * ((kBranch ? 1 : 0) + (kNext ? 1 : 0))) +
                   static_cast<int64_t>(group) * a.stages * N * row_bytes,
               bars + group * kMaxStages, a.stages, row_bytes};
  const auto start = [&](int stage, int64_t t) {
    const void* dr = a.dr != nullptr ? row_of(a.dr, a.lddr, t) : nullptr;
    if constexpr (kBranch && kNext)
      ring.start(stage, {dr, row_of(a.y, a.ldy, t), row_of(a.dn, a.lddn, t), row_of(a.r, a.ldr, t)});
    else if constexpr (kBranch) ring.start(stage, {dr, row_of(a.y, a.ldy, t)});
    else ring.start(stage, {dr, row_of(a.dn, a.lddn, t), row_of(a.r, a.ldr, t)});
  };
  if (kVec) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < 8 * kMaxStages; ++i) mbar_init(&bars[i], 1);
      fence_mbar_init();
      abort = 0;
    }
    __syncthreads();
    if (tid == 0)
      for (int k = 0; k < a.stages && row0 + k * groups < row1; ++k) start(k, row0 + k * groups);
  }
  if (kBranch) stage_weight(w, a.weight, a.H, padded);
  if (kNext) stage_weight(wn, a.next_weight, a.H, padded);
  __syncthreads();
  GroupSum sum{red, G, group, 0};
  const bool per_token = a.gate != nullptr && a.rows_per_gate == 0;
  const float* grow = a.gate != nullptr && !per_token ? a.gate + seg * a.H : nullptr;
  Eight acc_w[kChunks], acc_n[kChunks];
#pragma unroll
  for (int j = 0; j < kChunks; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc_w[j].p[i] = acc_n[j].p[i] = 0;
  const float inv_h = 1.f / a.H;
  const F2 alpha = pack2(a.alpha, a.alpha);
  // a row's own numbers are read a row ahead
  struct Scalars {
    float rstd_r, rstd_y, gate;
  };
  const auto scalars = [&](int64_t t) {
    return Scalars{kNext ? a.rstd_r[t] : 0.f, kBranch ? a.rstd_y[t] : 0.f, kBranch && per_token ? a.gate[t] : 1.f};
  };
  Scalars ahead{0.f, 0.f, 1.f};
  if (row0 < row1) ahead = scalars(row0);
  for (int64_t t = row0; t < row1; t += groups) {
    const Scalars own = ahead;
    if (t + groups < row1) ahead = scalars(t + groups);
    const auto get = [&](int array, const void* p, int64_t ld, const Places& at) {
      return kVec ? stage_chunk<E>(ring.array(array), at) : load_chunk<E, false>(row_of(p, ld, t), at);
    };
    if (kVec) ring.wait(a.status, &abort);
    Eight d[kChunks];
    if (kNext) {
      const float rstd = own.rstd_r;
      const F2 rs = pack2(rstd, rstd);
      F2 dot = 0;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const Places at = places<kVec>(tid, j, G, a.H);
        const Chunk<E> dn = get(kDn, a.dn, a.lddn, at), r = get(kR, a.r, a.ldr, at);
        const Eight wj = shared8<kVec>(wn, at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 rhat = mul2(r.pair(i), rs);
          acc_n[j].p[i] = fma2(dn.pair(i), rhat, acc_n[j].p[i]);
          d[j].p[i] = mul2(dn.pair(i), wj.p[i]);
          dot = fma2(d[j].p[i], rhat, dot);
        }
      }
      const float m = -sum(pair_sum(dot)) * inv_h * rstd;   // times r, not rhat, below
      const F2 mm = pack2(m, m);
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const Places at = places<kVec>(tid, j, G, a.H);
        const Chunk<E> r = get(kR, a.r, a.ldr, at);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[j].p[i] = mul2(rs, fma2(mm, r.pair(i), d[j].p[i]));
        if (a.dr != nullptr) {
          const Chunk<E> dr = get(kDr, a.dr, a.lddr, at);
#pragma unroll
          for (int i = 0; i < 4; ++i) d[j].p[i] = add2(d[j].p[i], dr.pair(i));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kChunks; ++j) d[j] = pairs(get(kDr, a.dr, a.lddr, places<kVec>(tid, j, G, a.H)));
    }
    Chunk<E> yr[kChunks];
    float s = 0.f;
    const float rstd_y = own.rstd_y, gt = own.gate;
    if (kBranch) {
      const F2 rs = pack2(rstd_y, rstd_y);
#pragma unroll
      for (int j = 0; j < kChunks; ++j) yr[j] = get(kY, a.y, a.ldy, places<kVec>(tid, j, G, a.H));
      // dx, and then d becomes v / gate
      F2 dot = 0;
      const F2 gg = pack2(gt, gt);
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const Places at = places<kVec>(tid, j, G, a.H);
        Eight v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v.p[i] = mul2(alpha, d[j].p[i]);
        store_chunk<E, kVec>(static_cast<E*>(a.dx) + t * a.H, at, v);
        const Eight wj = shared8<kVec>(w, at);
        Eight g;
        if (grow != nullptr) g = load_param<kVec>(grow, at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 yhat = mul2(yr[j].pair(i), rs);
          acc_w[j].p[i] = fma2(mul2(gg, d[j].p[i]), yhat, acc_w[j].p[i]);
          d[j].p[i] = mul2(d[j].p[i], wj.p[i]);
          if (grow != nullptr) d[j].p[i] = mul2(d[j].p[i], g.p[i]);
          dot = fma2(d[j].p[i], yhat, dot);
        }
      }
      s = sum(pair_sum(dot));   // the token gate's gradient; the mean below times the gate
    } else {
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        Eight v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v.p[i] = mul2(alpha, d[j].p[i]);
        store_chunk<E, kVec>(static_cast<E*>(a.dx) + t * a.H, places<kVec>(tid, j, G, a.H), v);
      }
      if (kVec) sum.sync();
    }
    if (kVec) {   // the group has read the row: its place is free
      if (G == 32) __syncwarp();
      if (tid == 0 && t + a.stages * groups < row1) start(ring.at, t + a.stages * groups);
      ring.next();
    }
    if (kBranch) {
      if (per_token && tid == 0) a.dgate_token[t] = s;
      const float m = -s * inv_h * rstd_y, f = rstd_y * gt;
      const F2 mm = pack2(m, m), ff = pack2(f, f);
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[j].p[i] = mul2(ff, fma2(mm, yr[j].pair(i), d[j].p[i]));
        store_chunk<E, kVec>(static_cast<E*>(a.dy) + t * a.H, places<kVec>(tid, j, G, a.H), d[j]);
      }
    }
  }
  // the groups' column sums, added in order, one row of the parts a CTA
  for (int which = 0; which < 2; ++which) {
    if (which == 0 ? !kBranch : !kNext) continue;
    float* out = (which == 0 ? a.part_w : a.part_n) + static_cast<int64_t>(blockIdx.x) * a.H;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const Places at = places<kVec>(tid, j, G, a.H);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = unpack2(which == 0 ? acc_w[j].p[i] : acc_n[j].p[i]);
        weights[group * padded + at.first + 2 * i * at.step] = v.x;
        weights[group * padded + at.first + (2 * i + 1) * at.step] = v.y;
      }
    }
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
  grid_dep_sync();   // launched beside the kernel that writes the sums
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

template <typename Args>
cudaError_t start(void (*kernel)(Args), std::atomic<bool>* smem_set, dim3 grid, int threads, size_t smem, cudaStream_t s,
                  const Args& a) {
  const cudaError_t e = set_smem_attr_once(smem_set, reinterpret_cast<const void*>(kernel), 208 * 1024);
  if (e != cudaSuccess) return e;
  kernel<<<grid, threads, smem, s>>>(a);
  return cudaGetLastError();
}

// Stages of a ring whose rows take `row` bytes a group: what `budget` bytes of shared memory leave, one at
// least (the largest: two weights of 8192 floats and four float32 rows, 192 KB).
int ring_stages(size_t weights, size_t row, int groups, size_t budget) {
  const size_t n = budget > weights ? (budget - weights) / (row * groups) : 0;
  return n < 1 ? 1 : n > kMaxStages ? kMaxStages : static_cast<int>(n);
}

template <typename E, bool kBranch, bool kNext>
cudaError_t forward_kernel(NormArgs& a, bool vec, cudaStream_t s) {
  static std::atomic<bool> set[2][64];
  const int threads = a.group > kNormThreads ? a.group : kNormThreads, groups = threads / a.group;
  const int64_t want = (a.T + groups - 1) / groups, most = static_cast<int64_t>(num_sms()) * (1024 / threads);
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  const size_t weights = sizeof(float) * 8 * kChunks * a.group * ((kBranch ? 1 : 0) + (kNext ? 1 : 0));
  if (!vec) return start(block_norm_kernel<E, kBranch, kNext, false>, set[0], grid, threads, weights, s, a);
  const size_t row = static_cast<size_t>(a.H) * sizeof(E) * (kBranch ? 2 : 1);
  // (32768 x 2048 BF16: one stage 88 us, two 91 us; wider rows have one in either case)
  a.stages = ring_stages(weights, row, groups, 36 * 1024);
  const size_t smem = weights + a.stages * row * groups;
  return start(block_norm_kernel<E, kBranch, kNext, true>, set[1], grid, threads, smem, s, a);
}

template <typename E>
cudaError_t forward(NormArgs a, cudaStream_t s) {
  const int e = sizeof(E);
  const bool vec = a.H % 8 == 0 && rows_aligned(a.x, a.ldx, e) && rows_aligned(a.y, a.ldy, e) &&
                   rows_aligned(a.r, a.H, e) && rows_aligned(a.n, a.H, e) &&
                   (a.rows_per_gate == 0 || rows_aligned(a.gate, a.H, 4));
  if (a.y == nullptr) return forward_kernel<E, false, true>(a, vec, s);
  return a.next_weight != nullptr ? forward_kernel<E, true, true>(a, vec, s) : forward_kernel<E, true, false>(a, vec, s);
}

template <typename E, bool kBranch, bool kNext>
cudaError_t backward_kernel(NormBackwardArgs& a, bool vec, int64_t segments, cudaStream_t s) {
  static std::atomic<bool> set[2][64];
  const int threads = a.group > kNormThreads ? a.group : kNormThreads, groups = threads / a.group;
  const dim3 grid(static_cast<unsigned>(segments * a.parts));
  const size_t unit = sizeof(float) * 8 * kChunks * a.group;
  const size_t weights = unit * ((kBranch ? 1 : 0) + (kNext ? 1 : 0));
  const size_t sums = unit * groups;   // the groups' column sums, at the end
  if (!vec)
    return start(block_norm_backward_kernel<E, kBranch, kNext, false>, set[0], grid, threads,
                 weights > sums ? weights : sums, s, a);
  const size_t row = static_cast<size_t>(a.H) * sizeof(E) * (1 + (kBranch ? 1 : 0) + (kNext ? 2 : 0));
  a.stages = ring_stages(weights, row, groups, threads > kNormThreads ? 200 * 1024 : 108 * 1024);   // 1 or 2 CTAs an SM
  const size_t smem = weights + a.stages * row * groups;
  return start(block_norm_backward_kernel<E, kBranch, kNext, true>, set[1], grid, threads, smem > sums ? smem : sums,
               s, a);
}

template <typename E>
cudaError_t backward(NormBackwardArgs a, int64_t segments, float* dweight, float* dgate, float* dnext,
                     cudaStream_t s) {
  const int e = sizeof(E);
  const bool vec = a.H % 8 == 0 && rows_aligned(a.dr, a.lddr, e) && rows_aligned(a.dn, a.lddn, e) &&
                   rows_aligned(a.r, a.ldr, e) && rows_aligned(a.y, a.ldy, e) && rows_aligned(a.dx, a.H, e) &&
                   rows_aligned(a.dy, a.H, e) && (a.rows_per_gate == 0 || rows_aligned(a.gate, a.H, 4));
  const bool next = a.next_weight != nullptr;
  const cudaError_t err = a.y == nullptr ? backward_kernel<E, false, true>(a, vec, segments, s)
                          : next         ? backward_kernel<E, true, true>(a, vec, segments, s)
                                         : backward_kernel<E, true, false>(a, vec, segments, s);
  if (err != cudaSuccess) return err;
  NormReduceArgs ra{a.part_w, a.part_n, a.weight, a.rows_per_gate > 0 ? a.gate : nullptr, a.H, segments, a.parts,
                    dweight, a.rows_per_gate > 0 ? dgate : nullptr, dnext};
  const int64_t blocks = (a.H + 31) / 32;
  return launch_pdl(true, block_norm_reduce_kernel,
                    dim3(static_cast<unsigned>(blocks * (2 + (ra.gate != nullptr ? segments : 0)))),
                    dim3(32 * kReduceSlices), 0, s, ra);
}

// Ranges of rows in all, unless there are more gate rows: the CTAs that 152 SMs hold (two an SM, one where a
// group is 512 threads).
int64_t norm_parts(int64_t H) { return group_threads(H) > kNormThreads ? 152 : 304; }

}  // namespace

int64_t block_norm_parts(int64_t T, int64_t gate_rows, int64_t H) {
  const int64_t segments = gate_rows > 0 ? gate_rows : 1, rows = T / segments;
  int64_t parts = norm_parts(H) / segments;
  if (parts > rows) parts = rows;
  return parts > 0 ? parts : 1;
}

cudaError_t launch_block_norm(const void* x, int64_t ldx, const void* y, int64_t ldy, int dtype, int64_t T, int64_t H,
                              const float* weight, const float* gate, int64_t gate_rows, float alpha,
                              const float* next_weight, float eps, void* r, void* n, float* rstd_y, float* rstd_r,
                              cudaStream_t s) {
  NormArgs a{x, y, ldx, ldy, T, static_cast<int>(H), group_threads(H), 1, weight, gate, next_weight,
             gate_rows > 0 ? T / gate_rows : 0, alpha, eps, r, n, rstd_y, rstd_r, device_status_ptr()};
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
  const int64_t segments = gate_rows > 0 ? gate_rows : 1, parts = block_norm_parts(T, gate_rows, H);
  NormBackwardArgs a{dr,     dn,    r,    y,    lddr,        lddn,
                     ldr,    ldy,   T,    static_cast<int>(H), group_threads(H), 1, rstd_y,
                     rstd_r, weight, gate, next_weight, gate_rows > 0 ? T / gate_rows : 0, alpha,
                     dx,     dy,    gate_rows > 0 ? nullptr : dgate, partial, partial + segments * parts * H,
                     T / segments, parts, device_status_ptr()};
  if (dtype == kActBF16) return backward<__nv_bfloat16>(a, segments, dweight, dgate, dnext, s);
  if (dtype == kActF16) return backward<__half>(a, segments, dweight, dgate, dnext, s);
  return backward<float>(a, segments, dweight, dgate, dnext, s);
}

}  // namespace nvfp4
