// Rows of logits over a vocabulary: loads of any alignment, and the one-pass softmax
// statistics that the token log probabilities and the distillation share.
//
// A row of V logits is cut into chunks of 8 consecutive elements by element number, and the
// chunks into vocab_slices(V) slices; thread i of a slice's 256 threads takes chunks i, i + 256,
// ... of the slice.  The cut depends on V alone -- not on the number of rows, not on whether
// the slices of a row run one after the other in one CTA or side by side in a cluster, and
// not on the row's address -- and so do a row's bits.
#pragma once
#include <cfloat>
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace nvfp4 {

constexpr int kVocabThreads = 256;
constexpr int kVocabWarps = kVocabThreads / 32;
constexpr int kMaxSlices = 8;
constexpr int kMaxList = 128;                 // top alternatives, teacher entries
constexpr int64_t kMaxVocab = 1 << 20;        // ids stay exact in the 20-bit parts of the kernels' keys
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A slice holds at least 4096 elements (two chunks a thread): smaller ones leave threads idle.
__host__ __device__ inline int vocab_slices(int64_t V) { return V >= 32768 ? 8 : V >= 16384 ? 4 : V >= 8192 ? 2 : 1; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- 8 elements at a time

__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 q;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "l"(p));
  return q;
}

template <typename E>
struct Chunk {
  static constexpr int kQ = sizeof(E) / 2;   // 16-byte words of 8 elements
  uint4 q[kQ];
};

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

__device__ __forceinline__ void unpack8(const Chunk<__nv_bfloat16>& c, float (&v)[8]) {
  const uint32_t w[4] = {c.q[0].x, c.q[0].y, c.q[0].z, c.q[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Chunk<__half>& c, float (&v)[8]) {
  const uint32_t w[4] = {c.q[0].x, c.q[0].y, c.q[0].z, c.q[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack8(const Chunk<float>& c, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(c.q[i].x);
    v[4 * i + 1] = __uint_as_float(c.q[i].y);
    v[4 * i + 2] = __uint_as_float(c.q[i].z);
    v[4 * i + 3] = __uint_as_float(c.q[i].w);
  }
}

// 8 elements that begin `shift` > 0 bytes into 16-byte words, word(0) the first.
template <int S, int N, int M>
__device__ __forceinline__ void funnel(const uint32_t (&w)[N], uint32_t (&o)[M], uint32_t bits) {
#pragma unroll
  for (int i = 0; i < M; ++i) o[i] = __funnelshift_r(w[i + S], w[i + S + 1], bits);
}
template <typename E, typename Word>
__device__ __forceinline__ Chunk<E> join_words(Word&& word, uint32_t shift) {
  constexpr int Q = Chunk<E>::kQ;
  uint32_t w[4 * Q + 5], o[4 * Q];
#pragma unroll
  for (int i = 0; i <= Q; ++i) {
    const uint4 q = word(i);
    w[4 * i] = q.x;
    w[4 * i + 1] = q.y;
    w[4 * i + 2] = q.z;
    w[4 * i + 3] = q.w;
  }
  w[4 * Q + 4] = 0;
  const uint32_t bits = (shift & 3u) * 8u;
  switch (shift >> 2) {
    case 0: funnel<0>(w, o, bits); break;
    case 1: funnel<1>(w, o, bits); break;
    case 2: funnel<2>(w, o, bits); break;
    default: funnel<3>(w, o, bits); break;
  }
  Chunk<E> r;
#pragma unroll
  for (int i = 0; i < Q; ++i) r.q[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  return r;
}

// One row and how to read it.  `shift` is the row's byte offset from a 16-byte boundary.
template <typename E>
struct Row {
  const E* p;
  int V;
  uint32_t shift;
  __device__ Row(const E* base, int64_t ld, int64_t row, int V_)
      : p(base + row * ld), V(V_), shift(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u) {}

  // Elements [8c, 8c + 8): one aligned read, or for a shifted row the 16-byte words around
  // them (all inside the row), joined by funnel shifts.  inner(c) says whether that is safe.
  __device__ __forceinline__ bool inner(int c) const {
    const int last = shift == 0 ? 8 * c + 8 : 8 * c + 8 + static_cast<int>((16 - shift) / sizeof(E));
    return last <= V && (shift == 0 || c > 0);
  }
  __device__ __forceinline__ Chunk<E> load_inner(int c) const {
    constexpr int Q = Chunk<E>::kQ;
    Chunk<E> r;
    const char* b = reinterpret_cast<const char*>(p + 8 * static_cast<int64_t>(c));
    if (shift == 0) {
#pragma unroll
      for (int i = 0; i < Q; ++i) r.q[i] = load16(b + 16 * i);
      return r;
    }
    return join_words<E>([&](int i) { return load16(b - shift + 16 * i); }, shift);
  }
  // Any chunk that begins inside the row; places past its end read as -inf (excluded).
  __device__ __forceinline__ void get(int c, float (&v)[8]) const {
    if (inner(c)) {
      unpack8(load_inner(c), v);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 8 * c + i < V ? to_f32(p[8 * c + i]) : -INFINITY;
  }
};

// ---------------------------------------------------------------- softmax statistics

// Over a set of logits z with c1 = scale * log2(e), t = (z - m) c1 and m their running
// maximum: s = sum 2^t and u = sum 2^t t.  m starts at the lowest float, so a set of -inf
// alone has s = 0 and a set of the lowest values is still uniform.  A NaN or +inf logit
// makes s (and u) NaN.
struct Stats {
  float m, s, u;
};
__device__ __forceinline__ Stats empty_stats() { return {-FLT_MAX, 0.f, 0.f}; }

template <bool kEntropy>
__device__ __forceinline__ void rebase(Stats& a, float m, float c1) {
  const float d = fmaxf((a.m - m) * c1, -1000.f);   // 2^-1000 is 0; keeps d * s away from inf * 0
  const float r = ex2(d);
  if (kEntropy) a.u = r * fmaf(d, a.s, a.u);
  a.s = r * a.s;
  a.m = m;
}
template <bool kEntropy>
__device__ __forceinline__ Stats merge(Stats a, Stats b, float c1) {
  const float m = fmaxf(a.m, b.m);
  rebase<kEntropy>(a, m, c1);
  rebase<kEntropy>(b, m, c1);
  a.s += b.s;
  if (kEntropy) a.u += b.u;
  return a;
}
template <bool kEntropy>
__device__ __forceinline__ float accumulate(Stats& a, const float (&v)[8], float c1) {
  float cm = v[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) cm = fmaxf(cm, v[i]);
  if (cm > a.m) rebase<kEntropy>(a, cm, c1);
  float s = 0.f, u = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = (v[i] - a.m) * c1;
    const float e = ex2(t);
    s += e;
    if (kEntropy) u = fmaf(e, fmaxf(t, -1000.f), u);   // an excluded token adds 0, not 0 * inf
  }
  a.s += s;
  if (kEntropy) a.u += u;
  return cm;
}
template <bool kEntropy>
__device__ __forceinline__ Stats warp_merge(Stats a, float c1) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stats b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.u = kEntropy ? __shfl_xor_sync(0xffffffffu, a.u, o) : 0.f;
    a = merge<kEntropy>(a, b, c1);
  }
  return a;
}

// The slices of a row join here: part[slice][warp], filled by every CTA of the row in the
// shared memory of the cluster's first CTA (or of each CTA).  Called by one warp; every lane
// returns the row's statistics.
template <bool kEntropy>
__device__ __forceinline__ Stats join_slices(const Stats (*part)[kVocabWarps], int slices, float c1) {
  const int lane = threadIdx.x & 31;
  const Stats* flat = &part[0][0];
  Stats a = lane < slices * kVocabWarps ? flat[lane] : empty_stats();
  if (lane + 32 < slices * kVocabWarps) a = merge<kEntropy>(a, flat[lane + 32], c1);
  return warp_merge<kEntropy>(a, c1);
}

// The chunks [first, last) of a slice.
__device__ __forceinline__ void slice_range(int V, int slices, int slice, int& first, int& last) {
  const int chunks = (V + 7) >> 3, per = (chunks + slices - 1) / slices;
  first = min(chunks, slice * per);
  last = min(chunks, first + per);
}

// Calls f(chunk number, 8 values) for this thread's chunks of [first, last), in order, with
// four loads in flight.
template <typename E, typename F>
__device__ __forceinline__ void for_chunks(const Row<E>& row, int first, int last, F&& f) {
  constexpr int kAhead = 4;
  int c = first + threadIdx.x;
  while (c < last) {
    const int end = c + (kAhead - 1) * kVocabThreads;
    if (end < last && row.inner(c) && row.inner(end)) {
      Chunk<E> raw[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) raw[i] = row.load_inner(c + i * kVocabThreads);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        float v[8];
        unpack8(raw[i], v);
        f(c + i * kVocabThreads, v);
      }
      c += kAhead * kVocabThreads;
    } else {
      float v[8];
      row.get(c, v);
      f(c, v);
      c += kVocabThreads;
    }
  }
}

// ---------------------------------------------------------------- stores

__device__ __forceinline__ void store_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_one(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// out[e] = f(e, value(e)) for e in [lo, hi) of a row, by `threads` threads of which this is
// number `tid`: eight(e, v) gives the values of [e, e + 8), one(e) a single one.  The chunks are
// cut on the output's 16-byte boundaries, so that stores are whole.
template <typename E, typename Eight, typename One, typename F>
__device__ __forceinline__ void map_chunks(E* out, int lo, int hi, int tid, int threads, Eight&& eight, One&& one,
                                           F&& f) {
  const uint32_t so = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(out + lo)) & 15u;
  const int head = min(hi - lo, static_cast<int>((16u - so) & 15u) / static_cast<int>(sizeof(E)));
  const int body = (hi - lo - head) >> 3;
  const int tail = lo + head + 8 * body;
  constexpr int kAhead = 2;
  for (int c = tid; c < body; c += kAhead * threads) {
    float v[kAhead][8];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (c + k * threads < body) eight(lo + head + 8 * (c + k * threads), v[k]);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int e = lo + head + 8 * (c + k * threads);
      if (c + k * threads < body) {
        f(e, v[k]);
        store8(out + e, v[k]);
      }
    }
  }
  // the ends, at most 7 elements each
  if (tid < head || (tid >= 8 && tid - 8 < hi - tail)) {
    const int e = tid < head ? lo + tid : tail + tid - 8;
    float v[8];
    v[0] = one(e);
#pragma unroll
    for (int i = 1; i < 8; ++i) v[i] = -INFINITY;
    f(e, v);
    store_one(out + e, v[0]);
  }
}

// The same with the values of z in global memory: z is read in whole words where it is aligned
// with the output, else one by one.  out may be z itself: a thread reads its elements before it
// writes them.
template <typename E, typename F>
__device__ __forceinline__ void map_range(const E* z, E* out, int lo, int hi, int tid, int threads, F&& f) {
  const bool same = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(z)) & 15u) == 0;
  map_chunks(
      out, lo, hi, tid, threads,
      [&](int e, float(&v)[8]) {
        if (same) {
          Chunk<E> c;
#pragma unroll
          for (int i = 0; i < Chunk<E>::kQ; ++i) c.q[i] = load16(reinterpret_cast<const char*>(z + e) + 16 * i);
          unpack8(c, v);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = to_f32(z[e + i]);
        }
      },
      [&](int e) { return to_f32(z[e]); }, f);
}

}  // namespace nvfp4
