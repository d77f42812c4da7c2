// Rows of logits over a vocabulary: loads of any alignment, and the one-pass softmax
// statistics that the token log probabilities and the distillation share.
//
// A row of V logits is cut into chunks of 8 consecutive elements by element number, and the
// chunks into vocab_slices(V) slices; thread i of a slice's 256 threads takes chunks i, i + 256,
// ... of the slice, four at a time (a batch).  The cut depends on V alone -- not on the number
// of rows, not on whether the slices of a row run one after the other in one CTA or side by
// side in a cluster, and not on the row's address -- and so do a row's bits.
//
// These kernels are bound by instructions as much as by HBM: at 6.8 TB/s an SM receives 11.7 BF16
// elements a cycle and issues 4 instructions for 32 lanes, so 11 an element are all it has.  So
// float32 arithmetic runs on pairs (add, mul and fma .f32x2), differences are taken from the 16-bit
// type, maxima on packed words, and the running maximum is met once a batch of 32 elements.
#pragma once
#include <cfloat>
#include <cooperative_groups.h>
#include <cstdint>
#include <type_traits>
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

// A slice holds at least 8192 elements, a batch of every thread: its sums are reduced over the warps once.
__host__ __device__ inline int vocab_slices(int64_t V) { return V >= 65536 ? 8 : V >= 32768 ? 4 : V >= 16384 ? 2 : 1; }

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

// Pairs of float32.
using F2 = uint64_t;
__device__ __forceinline__ F2 pack2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(F2 p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// What the kernels know of an element type: -inf in a packed word, the larger of two packed
// words, and the pairs and the maximum of a word.
template <typename E>
struct Packed;
template <>
struct Packed<__nv_bfloat16> {
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  static constexpr uint32_t kFar = 0xf149f149u;        // -1e30, twice
  static constexpr float kFarValue = -9.95e29f;        // a little above
  static __device__ __forceinline__ uint32_t clamp_far(uint32_t w) {   // at least kFar; NaN stays
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(kFar));
    return r;
  }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float minus(uint16_t h, float m) {   // h - m, h widened on the way
    float r;
    asm("sub.rn.f32.bf16 %0, %1, %2;" : "=f"(r) : "h"(h), "f"(m));
    return r;
  }
  static __device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
};
template <>
struct Packed<__half> {
  static constexpr uint32_t kNegInf = 0xfc00fc00u;
  static constexpr uint32_t kFar = 0xfbfffbffu;        // -65504, twice
  static constexpr float kFarValue = -65504.f;
  static __device__ __forceinline__ uint32_t clamp_far(uint32_t w) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(kFar));
    return r;
  }
  static __device__ __forceinline__ uint32_t max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float minus(uint16_t h, float m) {
    float r;
    asm("sub.rn.f32.f16 %0, %1, %2;" : "=f"(r) : "h"(h), "f"(m));
    return r;
  }
  static __device__ __forceinline__ float low(uint32_t w) { return __low2float(*reinterpret_cast<const __half2*>(&w)); }
  static __device__ __forceinline__ float high(uint32_t w) { return __high2float(*reinterpret_cast<const __half2*>(&w)); }
};

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

// 8 consecutive elements as they lie in memory.
template <typename E>
struct Chunk {
  static constexpr int kQ = sizeof(E) / 2;   // 16-byte words
  uint32_t w[4 * kQ];
  __device__ __forceinline__ void set(int i, uint4 q) {
    w[4 * i] = q.x;
    w[4 * i + 1] = q.y;
    w[4 * i + 2] = q.z;
    w[4 * i + 3] = q.w;
  }
  __device__ __forceinline__ F2 pair(int i) const {   // elements 2i, 2i + 1
    if constexpr (sizeof(E) == 4) return pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else return pack2(Packed<E>::low(w[i]), Packed<E>::high(w[i]));
  }
  __device__ __forceinline__ F2 pair_minus(int i, float m) const {   // the pair less m, rounded once
    if constexpr (sizeof(E) == 4) return add2(pair(i), pack2(-m, -m));
    else return pack2(Packed<E>::minus(static_cast<uint16_t>(w[i] & 0xffffu), m),
                      Packed<E>::minus(static_cast<uint16_t>(w[i] >> 16), m));
  }
  __device__ __forceinline__ float max() const {
    if constexpr (sizeof(E) == 4) {
      float m = __uint_as_float(w[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = fmaxf(m, __uint_as_float(w[i]));
      return m;
    } else {
      const uint32_t m = max_word();
      return fmaxf(Packed<E>::low(m), Packed<E>::high(m));
    }
  }
  __device__ __forceinline__ uint32_t max_word() const {
    return Packed<E>::max(Packed<E>::max(w[0], w[1]), Packed<E>::max(w[2], w[3]));
  }
  // element i (known at compile time) becomes -inf
  __device__ __forceinline__ void leave_out(int i) {
    if constexpr (sizeof(E) == 4) w[i] = 0xff800000u;
    else w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | (Packed<E>::kNegInf & 0xffff0000u)
                          : (w[i / 2] & 0xffff0000u) | (Packed<E>::kNegInf & 0xffffu);
  }
  __device__ __forceinline__ void put(int i, E v) {
    if constexpr (sizeof(E) == 4) w[i] = __float_as_uint(v);
    else {
      const uint32_t h = *reinterpret_cast<const uint16_t*>(&v);
      w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | (h << 16) : (w[i / 2] & 0xffff0000u) | h;
    }
  }
  __device__ __forceinline__ E get(int i) const {
    if constexpr (sizeof(E) == 4) return __uint_as_float(w[i]);
    else {
      const uint16_t h = static_cast<uint16_t>(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
      return *reinterpret_cast<const E*>(&h);
    }
  }
  static __device__ __forceinline__ Chunk none() {
    Chunk c;
#pragma unroll
    for (int i = 0; i < 4 * kQ; ++i) {
      if constexpr (sizeof(E) == 4) c.w[i] = 0xff800000u;
      else c.w[i] = Packed<E>::kNegInf;
    }
    return c;
  }
};
template <typename E>
__device__ __forceinline__ void unpack8(const Chunk<E>& c, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(c.pair(i));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
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
  for (int i = 0; i < 4 * Q; ++i) r.w[i] = o[i];
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
    const char* b = reinterpret_cast<const char*>(p + 8 * static_cast<int64_t>(c));
    if (shift == 0) {
      Chunk<E> r;
#pragma unroll
      for (int i = 0; i < Chunk<E>::kQ; ++i) r.set(i, load16(b + 16 * i));
      return r;
    }
    return join_words<E>([&](int i) { return load16(b - shift + 16 * i); }, shift);
  }
  // Any chunk that begins inside the row; places past its end read as -inf (excluded).
  __device__ __forceinline__ Chunk<E> get(int c) const {
    if (inner(c)) return load_inner(c);
    Chunk<E> r = Chunk<E>::none();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * c + i < V) r.put(i, p[8 * c + i]);
    return r;
  }
};

// ---------------------------------------------------------------- softmax statistics

// Over a set of logits z with c1 = scale * log2(e), t = (z - m) c1 and m their
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

// A thread's running sums: s and u of its even and odd elements.
template <typename E, bool kEntropy>
struct Running {
  float m = -FLT_MAX;
  F2 s = 0, u = 0;
  // Four chunks, 256 apart; only those of them that begin fewer than `left` chunks on count.
  // Returns their maximum.
  __device__ __forceinline__ float add(const Chunk<E> (&raw)[4], int left, float c1) {
    float cm;
    if constexpr (sizeof(E) == 4) {
      cm = raw[0].max();
#pragma unroll
      for (int k = 1; k < 4; ++k) cm = fmaxf(cm, k * kVocabThreads < left ? raw[k].max() : -INFINITY);
    } else {
      uint32_t w = raw[0].max_word();
#pragma unroll
      for (int k = 1; k < 4; ++k)
        w = Packed<E>::max(w, k * kVocabThreads < left ? raw[k].max_word() : Packed<E>::kNegInf);
      cm = fmaxf(Packed<E>::low(w), Packed<E>::high(w));
    }
    if (cm > m) {
      const float d = fmaxf((m - cm) * c1, -1000.f);
      const float r = ex2(d);
      const F2 rr = pack2(r, r);
      if (kEntropy) u = mul2(rr, fma2(pack2(d, d), s, u));
      s = mul2(rr, s);
      m = cm;
    }
    if constexpr (kEntropy && sizeof(E) == 2) {
      // Excluded tokens far below the maximum: as a far, finite value they add 0 to s and u, without a
      // clamp of every t.  2^-200 is 0; down to -1e38 every t is finite (0 * inf would be NaN).
      const float far = (Packed<E>::kFarValue - m) * c1;
      if (far < -200.f && far > -1e38f) {
        sum<true>(raw, left, c1);
        return cm;
      }
    }
    sum<false>(raw, left, c1);
    return cm;
  }
  template <bool kFar>
  __device__ __forceinline__ void sum(const Chunk<E> (&raw)[4], int left, float c1) {
    const F2 cc = pack2(c1, c1);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k > 0 && k * kVocabThreads >= left) break;
      Chunk<E> c = raw[k];
      if constexpr (kFar)
#pragma unroll
        for (int i = 0; i < 4; ++i) c.w[i] = Packed<E>::clamp_far(c.w[i]);
      F2 e[4];
      F2 x = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 tt = mul2(c.pair_minus(i, m), cc);
        const float2 t = unpack2(tt);
        e[i] = pack2(ex2(t.x), ex2(t.y));
        if (kEntropy) {   // an excluded token adds 0, not 0 * inf
          const F2 tu = kFar ? tt : pack2(fmaxf(t.x, -1000.f), fmaxf(t.y, -1000.f));
          x = i == 0 ? mul2(e[i], tu) : fma2(e[i], tu, x);
        }
      }
      s = add2(s, add2(add2(e[0], e[1]), add2(e[2], e[3])));
      if (kEntropy) u = add2(u, x);
    }
  }
  __device__ __forceinline__ Stats thread() const {
    const float2 ss = unpack2(s), uu = unpack2(u);
    return {m, ss.x + ss.y, kEntropy ? uu.x + uu.y : 0.f};
  }
  // The warp's statistics, the same in every lane.
  __device__ __forceinline__ Stats warp(float c1) const {
    return warp_join(thread(), c1);
  }
  // One after the other (in this order).
  static __device__ __forceinline__ Stats join(Stats a, Stats b, float c1) {
    const float m = fmaxf(a.m, b.m);
    rebase<kEntropy>(a, m, c1);
    rebase<kEntropy>(b, m, c1);
    a.s += b.s;
    if (kEntropy) a.u += b.u;
    return a;
  }
  static __device__ __forceinline__ Stats warp_join(Stats a, float c1) {
    rebase<kEntropy>(a, warp_top(a.m), c1);
    return warp_add(a);
  }
  // Of two sets a lane.
  static __device__ __forceinline__ Stats join_two(Stats a, Stats b, float c1) {
    const float m = warp_top(fmaxf(a.m, b.m));
    rebase<kEntropy>(a, m, c1);
    rebase<kEntropy>(b, m, c1);
    a.s += b.s;
    a.u += b.u;
    return warp_add(a);
  }
  static __device__ __forceinline__ float warp_top(float m) {
    float top;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(top) : "f"(m));
    return top;
  }
  static __device__ __forceinline__ Stats warp_add(Stats a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
      if (kEntropy) a.u += __shfl_xor_sync(0xffffffffu, a.u, o);
    }
    return a;
  }
  // The slices of a row join here: part[slice][warp], in the shared memory of the CTA.  Called by
  // one warp; every lane returns the row's statistics.
  static __device__ __forceinline__ Stats join_slices(const Stats (*part)[kVocabWarps], int slices, float c1) {
    const int lane = threadIdx.x & 31;
    const Stats* flat = &part[0][0];
    return join_two(lane < slices * kVocabWarps ? flat[lane] : empty_stats(),
                    lane + 32 < slices * kVocabWarps ? flat[lane + 32] : empty_stats(), c1);
  }
};

// Elements [lo, hi) of a row on their way from HBM into L2, in one request of one thread (whole 16-byte words).
template <typename E>
__device__ __forceinline__ void prefetch_row(const E* row, int lo, int hi) {
  const uintptr_t a = (reinterpret_cast<uintptr_t>(row + lo) + 15u) & ~uintptr_t(15);
  const uintptr_t b = reinterpret_cast<uintptr_t>(row + hi) & ~uintptr_t(15);
  if (a < b)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a), "r"(static_cast<uint32_t>(b - a)) : "memory");
}

// The chunks [first, last) of a slice.
__device__ __forceinline__ void slice_range(int V, int slices, int slice, int& first, int& last) {
  const int chunks = (V + 7) >> 3, per = (chunks + slices - 1) >> (__ffs(slices) - 1);   // 1, 2, 4 or 8 slices
  first = min(chunks, slice * per);
  last = min(chunks, first + per);
}

// Calls f(c, raw, last - c) for this thread's batches of [first, last), in order: raw[i] is
// chunk c + 256 i, and where that lies beyond the slice some chunk of it.  The four loads of a
// batch are in flight together.
template <typename E, typename F>
__device__ __forceinline__ void for_batches(const Row<E>& row, int first, int last, F&& f) {
  for (int c = first + threadIdx.x; c < last; c += 4 * kVocabThreads) {
    Chunk<E> raw[4];
    if (c + 3 * kVocabThreads < last && row.inner(c) && row.inner(c + 3 * kVocabThreads)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[i] = row.load_inner(c + i * kVocabThreads);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[i] = row.get(min(c + i * kVocabThreads, last - 1));
    }
    f(c, raw, last - c);
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

// out[e] = f(e, value(e)) for e in [lo, hi) of a row, by the first 256 threads: eight(e) gives the
// chunk of [e, e + 8), one(e) a single element, f(e, chunk, v) the eight results.  The chunks are
// cut on the output's 16-byte boundaries, so that stores are whole; kAhead of them are read
// before the first is written.
template <typename E, int kAhead, typename Eight, typename One, typename F>
__device__ __forceinline__ void map_chunks(E* out, int lo, int hi, Eight&& eight, One&& one, F&& f) {
  constexpr int kStep = 8 * kVocabThreads;
  const int tid = threadIdx.x;
  const uint32_t so = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(out + lo)) & 15u;
  const int head = min(hi - lo, static_cast<int>((16u - so) & 15u) / static_cast<int>(sizeof(E)));
  const int base = lo + head, tail = base + ((hi - base) & ~7);
  const auto some = [&](int e, auto n) {
    constexpr int N = decltype(n)::value;
    Chunk<E> raw[N];
#pragma unroll
    for (int k = 0; k < N; ++k) raw[k] = eight(e + k * kStep);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float v[8];
      f(e + k * kStep, raw[k], v);
      store8(out + e + k * kStep, v);
    }
  };
  int e = base + 8 * tid;
  for (; e + (kAhead - 1) * kStep < tail; e += kAhead * kStep) some(e, std::integral_constant<int, kAhead>());
  if (kAhead > 1)
    for (; e < tail; e += kStep) some(e, std::integral_constant<int, 1>());
  // the ends, at most 7 elements each
  if (tid < head || (tid >= 8 && tid - 8 < hi - tail)) {
    const int at = tid < head ? lo + tid : tail + tid - 8;
    Chunk<E> c = Chunk<E>::none();
    c.put(0, one(at));
    float v[8];
    f(at, c, v);
    store_one(out + at, v[0]);
  }
}

// The same with the values in the row z[0, V) of global memory.  Where z and out are not
// equally far from a 16-byte boundary, z's words are joined by funnel shifts (inside the
// row; its ends are read one by one).  out may be z itself: a thread then reads its own
// elements alone, before it writes them.
template <typename E, int kAhead, typename F>
__device__ __forceinline__ void map_row(const E* z, int V, E* out, int lo, int hi, F&& f) {
  constexpr int Q = Chunk<E>::kQ;
  const auto one = [&](int e) { return z[e]; };
  // the shift of every chunk: out + e is on a boundary
  const uint32_t shift =
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z) - reinterpret_cast<uintptr_t>(out)) & 15u;
  if (shift == 0) {
    map_chunks<E, kAhead>(
        out, lo, hi,
        [&](int e) {
          Chunk<E> c;
#pragma unroll
          for (int i = 0; i < Q; ++i) c.set(i, load16(reinterpret_cast<const char*>(z + e) + 16 * i));
          return c;
        },
        one, f);
    return;
  }
  const int before = shift / sizeof(E), after = static_cast<int>((16 - shift) / sizeof(E));
  map_chunks<E, 2>(
      out, lo, hi,
      [&](int e) {
        if (e >= before && e + 8 + after <= V)
          return join_words<E>(
              [&](int i) { return load16(reinterpret_cast<const char*>(z + e) - shift + 16 * i); }, shift);
        Chunk<E> c = Chunk<E>::none();
#pragma unroll
        for (int i = 0; i < 8; ++i) c.put(i, z[e + i]);
        return c;
      },
      one, f);
}

}  // namespace nvfp4
