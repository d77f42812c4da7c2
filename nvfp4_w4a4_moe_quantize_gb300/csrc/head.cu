// Log probabilities straight from hidden rows and the head's weight, and their gradients: the
// softmax cross entropy over a large vocabulary without its logits in memory.
//
// c_tj = scale <hidden_t, weight_j>;  lse_t = ln sum_j exp(c_tj);  p_tj = exp(c_tj - lse_t);
// logprob_t = c_ty - lse_t;  entropy_t = -sum_j p_tj ln p_tj.  The gradient by c is
// d_tj = dlogprob_t (1[j = y] - p_tj) - dentropy_t p_tj (ln p_tj + entropy_t), and
// dhidden = scale d weight, dweight = scale d^T hidden.
//
// Forward: one product whose epilogue keeps of every row and 128 columns the largest logit, the
// sum of exponentials below it and (entropy) their weighted sum; a second kernel joins them.
// The columns of a partial result are fixed by V, so a row's bits depend on its hidden row, the
// weight and scale alone, not on the other rows.
// Backward: the vocabulary in pieces.  Of a piece the logits are computed again and turned into
// d (16 bits, [rows, piece] in the workspace); then dhidden += d weight (float32 sums over the
// pieces) and the piece of dweight = d^T hidden in one launch.  Rows without a token to score take
// no part: the others are gathered first.
//
// One kernel runs the three products.  Roles: warp 0 loads (TMA, 64 x 64 boxes of 128-byte rows,
// 128-byte swizzle), warp 1 issues the MMAs (tcgen05, float32 accumulators of 256 columns in
// TMEM, two of them, so the epilogue of one tile runs under the products of the next), warps 2-9
// are the epilogue: a thread has one row and 128 of the tile's 256 columns.  More than 128 rows run by
// pairs of CTAs (M = 256, N = 256: 64 KB of operands for 2^22 products), fewer by single ones.
//
// Measured, 8192 x 131072 x 2048 BF16 with a tenth of the rows ignored: forward 2.32-2.34 ms, 1.69-1.71 PF/s, backward
// 7.49-7.59 ms, 1.56-1.58 PF/s; a library product holds 1.74 under the same power limit.  Bound by the tensor cores and, a
// little behind them, by what precision asks of the epilogue: the logits' stretches (2.25 ms in one), the long products'
// (7.28 ms without) and what the rounding of the targets' d left.  One row: 101-102 us, the weight at 5.8 TB/s.  The
// statistics and d hold 128 logits a thread at 168 registers, the most that ten warps allow, and spill some 10 of their
// other values (24-52 bytes).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "pdl.cuh"
#include "ptx.cuh"
#include "vocab.cuh"

namespace nvfp4 {
namespace {

constexpr int kBM = 128;                 // rows of a CTA's tile (one a TMEM lane)
constexpr int kBK = 64;                  // a block of the contraction: one 128-byte swizzle row of 16-bit values
constexpr int kBox = 64 * 128;           // bytes of one 64 x 64 box
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kPart = 128;               // columns of a partial result, and of a thread of the epilogue
constexpr float kLowestLse = -16777216.f;

enum : int { kStats = 0, kGrad = 1, kProducts = 2 };

// Logits are summed in stretches of at most 512 products.  A tensor core adds 16 products at a time and cuts off
// what lies below the largest of them and of the sum, always towards zero, so the error of a long sum grows with its
// length (measured: sums of one sign lose 2.4 units in the last place a step, sums of random signs a quarter); the
// stretches are added to one another in registers, rounded to nearest.  H = 2048, relative errors of lse / entropy and the
// time of 8192 x 131072 logits: one stretch 6e-7 / 1.1e-6, 2.25 ms; 1024: 3e-7 / 5e-7, 2.24 ms; 512: 1.5e-7 / 2.4e-7,
// 2.34 ms; a float32 product 0.9e-7 / 5e-7.  (An accumulator takes some 4000 cycles to read under running MMAs, so
// shorter stretches wait for it: 256 at H = 1024 takes 770 us of 8192 x 65536 logits, 512 609, 1024 571.)  A single
// row's log probability, 12 inputs of H = 2048: up to 1.7e-6 off with 1024, 7e-7 with 512.
constexpr int kStretch = 512 / kBK;

// The gradients' products, as long as the vocabulary or the batch, go in stretches of at most 8192, added in float32
// through a part of the workspace that stays in L2 (a thread reads its own numbers again).  A single sum of 131072
// lost 2.6e-4 of a target's w_y, where half precision's own rounding is 2.4e-4; in stretches 2e-5.  8192 x 131072 x 2048,
// four of them a tile of dhidden: 7.28 -> 7.42 ms; stretches of 16384 7.40, of 4096 7.74.
constexpr int kLong = 8192 / kBK;
constexpr int kMaxCtas = 152;            // a GB300's SMs; the grid is no larger
constexpr size_t kLongBytes = (size_t)kEpiWarps * 32 * 128 * 4;   // of a CTA

// Columns of a tile: 256; 128 for the logits of few rows by single CTAs, which the weight's bytes bound: the
// smaller tiles spread more evenly over the SMs (96 x 50021 x 1032: 30 us against 34).
constexpr int tile_cols(int mode, bool pair) { return pair || mode == kProducts ? 256 : 128; }

template <int kMode, bool kPair>
struct Ring {
  static constexpr int kBN = tile_cols(kMode, kPair);
  static constexpr int kABoxes = 2;                                    // 128 rows of A
  static constexpr int kBBoxes = (kPair ? kBN / 2 : kBN) / 64;         // B's rows, or this CTA's half of them
  // A stage is two blocks of the contraction, with one barrier each way: against stages of one block it raised
  // the tensor cores' share of the time from 84 to 98% (8192 x 131072 x 2048).
  static constexpr int kSub = 2;
  static constexpr int kSubBytes = (kABoxes + kBBoxes) * kBox;
  static constexpr int kStageBytes = kSub * kSubBytes;
  static constexpr int kStages = kBBoxes == 2 ? 3 : 2;
  // The epilogue's warps.  256 columns: each has half of every tile, of two accumulators; 128: warps 0-3 and
  // 4-7 take turns with the tiles, each four with two accumulators of their own.
  static constexpr int kGroups = kBN == 256 ? 1 : 2;
  static constexpr int kAccWarps = kEpiWarps / kGroups;
  static constexpr int kAccs = 2 * kGroups;
};

template <int kMode, bool kPair>
struct HeadSmem {
  using R = Ring<kMode, kPair>;
  uint8_t stage[R::kStages][R::kStageBytes];
  uint8_t out[kEpiWarps][32 * 128];      // boxes of dweight on their way out
  uint64_t full[R::kStages];
  uint64_t empty[R::kStages];
  uint64_t accf[R::kAccs];
  uint64_t acce[R::kAccs];
  uint64_t fin;
  uint32_t tmem_base;
  int abort;
};
template <int kMode, bool kPair>
constexpr size_t smem_bytes() { return sizeof(HeadSmem<kMode, kPair>) + 1024; }
static_assert(smem_bytes<kStats, false>() <= 232448 && smem_bytes<kProducts, false>() <= 232448 &&
                  smem_bytes<kProducts, true>() <= 232448,
              "shared memory budget");

// d travels in 16 bits.  A gradient hangs on the targets' d above all, so what their rounding leaves is kept in
// float32, one number a row: dhidden gains it times the target's weight where its sums are rounded, dweight times the
// hidden row in the epilogue of the target's tile (a list of blocks of 32 rows for every 32 tokens says where).  Errors
// of both gradients against the result's own rounding, logits of deviation 2, 65 to 600 rows: 1.4 times, on single
// inputs 1.6, without it; 1.00-1.01 with it.  8192 x 131072 x 2048 7.49 -> 7.55 ms, 1001 x 50021 x 1032 231 -> 246 us,
// 96 x 131072 x 2048 308 -> 335 us (the epilogue's instructions bound few rows).  One warp adds up what 32 tokens gain,
// some 200 cycles a row where many have targets there: 8.4 ms against 8.05 where 32 tokens have two fifths of the 8192 rows,
// at 32768 x 32768 x 1024 7.2 against 4.5 (four rows' loads at a time 8.7 and 8.6).  A kernel of its own for it: 8.4 and 6.0 ms
// there, but 261 us at 1001 rows, 354 at 96, 5.0 ms with targets at random.
// Of up to 64 rows all of d is held as two 16-bit numbers, the rounded value and what the rounding left: single
// values other than the targets' show there as well.  The second numbers are rows of their own behind the first ones',
// the hidden rows are repeated for them; both products are bound by the weight's bytes, and 48 x 131072 x 2048 takes 310 us
// against 287 with one number (96 and 128 rows, which fill two tiles, 400 and 418 us; 256 rows by pairs 375).
constexpr int kTwoParts = 64;

// What a row of the gradient needs: d = p (a + b log2 p), + zy at the target.
struct RowGrad {
  float a, b, lse, zy;
};

struct HeadArgs {
  int64_t T;                 // rows of `hidden`
  const int32_t* n_rows;     // rows that take part, nullable: T
  bool always_gathered;      // the gathered rows are read even if all of them take part (products, half precision)
  int V, H;
  int f16;
  float scale;
  int* status;
  int x_rows;                // rows of a box of hidden rows: 64, or fewer where there are no more
  // statistics
  const int32_t* targets;    // nullable
  const int32_t* index;      // row -> row of targets, nullable: itself
  float* part_m;             // [parts][pitch]
  float* part_s;
  float* part_u;             // nullable: no entropy
  int64_t pitch;
  float* target_logit;       // [rows], unscaled
  // gradient
  int v0, width;             // the piece of the vocabulary
  const RowGrad* rows;
  const int32_t* row_target;
  bool entropy;              // some row's b is not 0
  int low;                   // rows from a number of d to its second part (a multiple of 16), or 0: there is none
  float* left;               // [rows]: what the rounding of the target's d left, nullable (d has two parts)
  uint16_t* d_out;           // [rows][d_pitch]
  int64_t d_pitch;
  // products
  float* long_sums;          // [CTAs][kLongBytes]: of a tile's earlier stretches; null: one stretch each
  float* x_sums;             // [x_splits][x_pitch][H]
  int x_splits;              // parts of dhidden's contraction
  int64_t x_pitch;           // rows between their sums
  bool x_first;              // the first piece stores, the others add
  bool want_x, want_w;
  const float* w_factor;     // nullable: 1
  const uint32_t* marks;     // [V / 32][mark_words]: blocks of 32 rows with a target among 32 tokens; with `left`
  int mark_words;
  const void* x_all;         // hidden rows as they are, and gathered (or weighted)
  int64_t x_all_ld;
  const void* x_gathered;
  int64_t x_gathered_ld;
  float* fixes;              // [CTAs][kLongBytes]: what targets add to a tile
};

__device__ __forceinline__ uint32_t idesc_16(bool f16, uint32_t M, uint32_t N, bool a_mn, bool b_mn) {
  const uint32_t fmt = f16 ? 0u : 1u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((N >> 3) << 17) | ((M >> 4) << 24);
}

// One tile of work.
struct Unit {
  bool w;                    // products: a tile of dweight (else of dhidden)
  int m, n, split;           // tile numbers (m in CTA-pair rows where there are pairs)
  int cols;                  // columns to compute: a multiple of 32
  int k0, k1;                // stages of the contraction
  int turns, len;            // stretches, stages of one (the last may be shorter)
};

// The tiles of one CTA or pair, unit(0), unit(1), ... until it says false.
template <int kMode, bool kPair>
struct Plan {
  static constexpr int kBN = tile_cols(kMode, kPair);
  static constexpr int kTileM = kPair ? 2 * kBM : kBM;
  int p, P;                  // this one, of how many
  int m_tiles, n_tiles, total;
  // products: the kind with the longer contraction goes first, one after the other to everyone; those
  // who got one less take more of the other kind
  bool x_long;
  int xm, xn, x_kb, w_kb, longs, shorts, extra, both, more;
  __device__ Plan(const HeadArgs& a, int n) {
    p = kPair ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    P = kPair ? (int)(gridDim.x >> 1) : (int)gridDim.x;
    if (kMode == kProducts) {
      xm = (n + kTileM - 1) / kTileM;
      xn = (a.H + kBN - 1) / kBN;
      x_kb = (a.width + kBK - 1) / kBK;
      w_kb = ((n > 0 ? n + a.low : 0) + kBK - 1) / kBK;
      const int xs = a.want_x ? xm * xn * a.x_splits : 0, ws = a.want_w ? (a.width + kTileM - 1) / kTileM * xn : 0;
      // a tile's cost in stages of the contraction, its epilogue as 8
      const int cx = x_kb / a.x_splits + 8, cw = w_kb + 8;
      x_long = cx >= cw;
      longs = x_long ? xs : ws;
      shorts = x_long ? ws : xs;
      extra = longs % P;                           // the first `extra` have one long tile more
      const int ratio = x_long ? cx / cw : cw / cx;
      // `both` short tiles for everyone, `more` for those without a long one more
      more = extra > 0 ? ratio : 0;
      if ((int64_t)more * (P - extra) >= shorts) {
        both = 0;
        more = extra > 0 ? (shorts + P - extra - 1) / (P - extra) : 0;
      } else {
        both = (shorts - more * (P - extra) + P - 1) / P;
      }
    } else {
      m_tiles = (n + kTileM - 1) / kTileM;
      n_tiles = (a.width + kBN - 1) / kBN;
      total = m_tiles * n_tiles;
    }
  }
  __device__ bool unit(const HeadArgs& a, int i, Unit& u) const {
    u = Unit{};
    if (kMode != kProducts) {
      const int t = p + i * P;
      if (t >= total) return false;
      u.n = t / m_tiles;                 // the weight's rows are read once, the hidden rows stay in L2
      u.m = t - u.n * m_tiles;
      u.cols = kBN;
      u.k1 = (a.H + kBK - 1) / kBK;
      u.turns = (u.k1 + kStretch - 1) / kStretch;
      constexpr int kSub = Ring<kMode, kPair>::kSub;
      u.len = ((u.k1 + u.turns - 1) / u.turns + kSub - 1) / kSub * kSub;   // whole stages
      u.turns = (u.k1 + u.len - 1) / u.len;
      return true;
    }
    int t;
    const int mine = longs / P + (p < extra ? 1 : 0);
    const bool first = i < mine;
    if (first) {
      t = p + i * P;
    } else {
      i -= mine;
      if (i < both) {
        t = p + i * P;
      } else {
        i -= both;
        if (p < extra || i >= more) return false;
        t = both * P + i * (P - extra) + p - extra;
      }
      if (t >= shorts) return false;
    }
    u.w = first != x_long;
    if (!u.w) {
      const int per = xm * xn;
      u.split = t / per;
      t -= u.split * per;
      u.k0 = (int)((int64_t)x_kb * u.split / a.x_splits);
      u.k1 = (int)((int64_t)x_kb * (u.split + 1) / a.x_splits);
    } else {
      u.k1 = w_kb;
    }
    u.m = t / xn;
    u.n = t - u.m * xn;
    u.cols = min(kBN, (a.H - u.n * kBN + 31) / 32 * 32);
    const int span = u.k1 - u.k0;
    u.turns = a.long_sums != nullptr ? max((span + kLong - 1) / kLong, 1) : 1;
    constexpr int kSub = Ring<kMode, kPair>::kSub;
    u.len = ((span + u.turns - 1) / u.turns + kSub - 1) / kSub * kSub;   // whole stages
    return true;
  }
};

// 32 bytes a thread: whole sectors, whatever the other rows' threads do.  (d through shared memory and TMA
// stores: 87% of the cycles with the tensor cores active against 92; dweight, whose tiles are shorter, the other way.)
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void load32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_16bit(float lo, float hi, int f16) {
  uint32_t w;
  if (f16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

__device__ __forceinline__ float2 unpack_16bit(uint32_t w, int f16) {
  if (f16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// kMany: products whose contractions have several stretches; kLeft: dweight with what the rounding of the targets' d
// left.  (Asked of every tile they slowed those that have neither: 335 and 341 us against 311 at 48 x 131072 x 2048.)
template <int kMode, bool kPair, bool kMany, bool kLeft>
__global__ void __launch_bounds__(kThreads, 1)
    head_kernel(const __grid_constant__ CUtensorMap hidden, const __grid_constant__ CUtensorMap gathered,
                const __grid_constant__ CUtensorMap weight, const __grid_constant__ CUtensorMap dlogits,
                const __grid_constant__ CUtensorMap dweight, const HeadArgs a) {
  using R = Ring<kMode, kPair>;
  constexpr int kStages = R::kStages, kBN = R::kBN;
  extern __shared__ uint8_t smem_raw[];
  using Smem = HeadSmem<kMode, kPair>;
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int i = 0; i < R::kAccs; ++i) {
      mbar_init(&sm.accf[i], 1);
      mbar_init(&sm.acce[i], kPair ? 2 * R::kAccWarps : R::kAccWarps);
    }
    mbar_init(&sm.fin, 1);
    sm.abort = 0;
    fence_mbar_init();
    prefetch_tensormap(&weight);
    prefetch_tensormap(kMode == kProducts ? &dlogits : &hidden);
  }
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(&sm.tmem_base, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&sm.tmem_base, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();   // both CTAs' barriers exist before any remote arrival
  tc_fence_after();
  grid_dep_sync();
  fence_proxy_async_global();   // the loads read what the last kernels' threads wrote
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;
  // Loads and MMAs complete the other barriers (the async proxy); `acce` hears from a pair's other CTA's threads.
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, a.status, abort); };
  auto wait_acce = [&](uint64_t* bar, uint32_t parity) {
    return kPair ? mbar_wait_cluster(bar, parity, a.status, abort) : mbar_wait(bar, parity, a.status, abort);
  };
  const int n_rows = a.n_rows != nullptr ? *a.n_rows : (int)a.T;
  const Plan<kMode, kPair> plan(a, n_rows);
  constexpr int kTileM = kPair ? 2 * kBM : kBM;

  if (warp == 0) {
    if (lane == 0) {
      const CUtensorMap* x = a.always_gathered || n_rows < a.T ? &gathered : &hidden;
      uint32_t stage = 0, phase = 0;
      Unit u;
      for (int t = 0; plan.unit(a, t, u); ++t) {
        const int am = u.m * kTileM + (int)rank * kBM;                       // this CTA's rows of A
        const int bn = u.n * kBN + (kPair ? (int)rank * (u.cols / 2) : 0);   // and of B
        for (int i = 0; i < u.turns; ++i) {
          const int kb1 = min(u.k0 + (i + 1) * u.len, u.k1);
          for (int kb0 = u.k0 + i * u.len; kb0 < kb1; kb0 += R::kSub) {
            if (!wait(&sm.empty[stage], phase ^ 1u)) goto loads_done;
            const int subs = min(R::kSub, kb1 - kb0);
            // a pair's bytes all count on CTA 0's barrier
            // one box of A where there are no more rows
            const int a_boxes = !kPair && (kMode == kProducts ? !u.w && a.low > 0 && a.low <= 32 : a.T <= 64) ? 1 : R::kABoxes;
            const uint32_t bytes = subs * (R::kBBoxes * kBox + a_boxes * (kMode != kProducts ? a.x_rows * 128 : kBox));
            if (rank == 0) mbar_arrive_expect_tx(&sm.full[stage], (kPair ? 2 : 1) * bytes);
            const uint32_t bar = kPair ? cluster_addr(&sm.full[stage], 0) : smem_u32(&sm.full[stage]);
            for (int sub = 0; sub < subs; ++sub) {
              uint8_t* dst = sm.stage[stage] + sub * R::kSubBytes;
              auto load = [&](int box, const CUtensorMap* map, int cx, int cy) {
                if (kPair) tma_load_2d_pair(dst + box * kBox, map, cx, cy, bar);
                else tma_load_2d(dst + box * kBox, map, cx, cy, &sm.full[stage]);
              };
              const int k = (kb0 + sub) * kBK;
              if (kMode != kProducts) {
#pragma unroll
                for (int i = 0; i < R::kABoxes; ++i)
                  if (i < a_boxes) load(i, x, k, am + 64 * i);
#pragma unroll
                for (int i = 0; i < R::kBBoxes; ++i) load(R::kABoxes + i, &weight, k, a.v0 + bn + 64 * i);
              } else if (!u.w) {
#pragma unroll
                for (int i = 0; i < R::kABoxes; ++i)
                  if (i < a_boxes) load(i, &dlogits, k, am + 64 * i);
#pragma unroll
                for (int i = 0; i < R::kBBoxes; ++i) load(R::kABoxes + i, &weight, bn + 64 * i, a.v0 + k);
              } else {
#pragma unroll
                for (int i = 0; i < R::kABoxes; ++i) load(i, &dlogits, am + 64 * i, k);
#pragma unroll
                for (int i = 0; i < R::kBBoxes; ++i) load(R::kABoxes + i, x, bn + 64 * i, k);
              }
            }
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
    loads_done:;
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      const uint32_t st0 = smem_u32(sm.stage[0]);
      constexpr uint32_t kStageDesc = R::kStageBytes >> 4;
      const uint64_t a_k = smem_desc(st0, 16, 1024, 2), b_k = smem_desc(st0 + R::kABoxes * kBox, 16, 1024, 2);
      const uint64_t a_m = smem_desc(st0, kBox, 1024, 2), b_m = smem_desc(st0 + R::kABoxes * kBox, kBox, 1024, 2);
      // Whether the next stage has arrived is asked before this stage's MMAs are issued: the answer is there when
      // it is needed.
      uint32_t stage = 0, phase = 0;
      bool full_ready = false;
      Unit u;
      uint32_t turn[R::kGroups] = {};
      bool more = plan.unit(a, 0, u);
      for (int it = 0; more;) {
        const bool a_mn = kMode == kProducts && u.w, b_mn = kMode == kProducts;
        const uint32_t idesc = idesc_16(a.f16 != 0, kTileM, u.cols, a_mn, b_mn);
        // K-major: a step of 16 is 32 bytes of each row.  Other-major: a box is 64 rows of the
        // contraction by 64 columns; a step is 16 rows (2048 bytes), the next 64 columns one box on.
        const uint64_t a0 = a_mn ? a_m : a_k, b0 = b_mn ? b_m : b_k;
        const uint32_t a_step = a_mn ? 128 : 2, b_step = b_mn ? 128 : 2;
        const int k1 = u.k1, len = u.len, turns = u.turns, group = R::kGroups == 1 ? 0 : it & 1;
        int kb = u.k0;
        more = plan.unit(a, ++it, u);   // the next tile, while this one's products run
        for (int i = 0; i < turns; ++i) {
          const uint32_t n = turn[R::kGroups == 1 ? 0 : group]++;
          const uint32_t acc = 2 * group + (n & 1), d = tmem + acc * kBN;
          if (!wait_acce(&sm.acce[acc], ((n >> 1) & 1) ^ 1u)) goto mma_done;
          tc_fence_after();
          const int kb0 = kb;
          kb = min(kb0 + len, k1);
          for (int b = kb0; b < kb; b += R::kSub) {
            if (!full_ready && !wait(&sm.full[stage], phase)) goto mma_done;
            const uint64_t ad = a0 + stage * kStageDesc, bd = b0 + stage * kStageDesc;
            uint64_t* const empty = &sm.empty[stage];
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
            full_ready = mbar_test(&sm.full[stage], phase);
#pragma unroll
            for (int sub = 0; sub < R::kSub; ++sub) {
              if (b + sub >= kb) break;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                constexpr uint32_t kNext = R::kSubBytes >> 4;
                const uint64_t as = ad + sub * kNext + a_step * j, bs = bd + sub * kNext + b_step * j;
                const uint32_t on = b > kb0 || sub + j > 0 ? 1u : 0u;
                if (kPair) tc_mma_f16_pair(d, as, bs, idesc, on);
                else tc_mma_f16(d, as, bs, idesc, on);
              }
            }
            if (kPair) tc_commit_pair_both(empty);
            else tc_commit(empty);
          }
          if (kPair) tc_commit_pair_both(&sm.accf[acc]);
          else tc_commit(&sm.accf[acc]);
        }
      }
    mma_done:
      // whatever the exit, no MMA is still running when the TMEM is freed (a bounded wait of its
      // own, also after an abort)
      if (kPair) tc_commit_pair(cluster_addr(&sm.fin, 0));
      else tc_commit(&sm.fin);
      volatile int no_abort = 0;
      mbar_wait(&sm.fin, 0, a.status, &no_abort, 1000000000ull);
    }
  } else {
    const int q = warp & 3, ew = warp - 2;                   // q: the TMEM lanes that this warp may read
    const int half = R::kGroups == 1 ? ew >> 2 : 0, group = R::kGroups == 1 ? 0 : ew >> 2;
    const uint32_t acce0 = kPair ? cluster_addr(&sm.acce[0], 0) : 0u;
    uint8_t* buf = sm.out[ew];
    const float c1 = a.scale * kLog2e;
    auto release = [&](uint32_t acc) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kPair) mbar_arrive_cluster(acce0 + acc * (uint32_t)sizeof(uint64_t));
        else mbar_arrive(&sm.acce[acc]);
      }
    };
    uint32_t turn = 0;
    Unit u;
    for (int it = 0; plan.unit(a, it, u); ++it) {
      if (R::kGroups == 2 && (it & 1) != group) continue;
      const int row0 = u.m * kTileM + (int)rank * kBM + q * 32, row = row0 + lane;
      const int col0 = u.n * kBN + half * 128;
      uint32_t v[kMode == kProducts ? 2 : 4][32];
      if constexpr (kMode != kProducts) {
        // the logits of this thread's 128 columns, the same bits in both kernels
        bool ready = true;
        for (int i = 0; i < u.turns; ++i) {
          const uint32_t acc = 2 * group + (turn & 1);
          ready = __all_sync(0xFFFFFFFFu, wait(&sm.accf[acc], (turn >> 1) & 1));
          if (!ready) break;
          ++turn;
          tc_fence_after();
          const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + acc * kBN + half * 128;
          if (i == 0) {
#pragma unroll
            for (int c = 0; c < 4; ++c) NVFP4_TMEM_LD_X32(taddr + 32 * c, v[c]);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_loaded(v[c]);
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint32_t w[16];
              NVFP4_TMEM_LD_X16(taddr + 16 * c, w);
              tmem_ld_wait();
              tmem_loaded(w);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                uint32_t& x = v[c >> 1][(c & 1) * 16 + j];
                x = __float_as_uint(__uint_as_float(x) + __uint_as_float(w[j]));
              }
            }
          }
          release(acc);
        }
        if (!ready) break;
      }
      if constexpr (kMode == kStats) {
        int rel = -1;                                          // the target's place among this thread's columns
        if (a.targets != nullptr && row < n_rows)
          rel = a.targets[a.index != nullptr && n_rows < a.T ? a.index[row] : row] - col0;
        auto val = [&](int i) { return __uint_as_float(v[i >> 5][i & 31]); };
        const int live = min(max(a.width - col0, 0), 128);
        if (live < 128) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i >= live) v[i >> 5][i & 31] = 0xFF800000u;   // -inf
        }
        if (row0 >= n_rows || live == 0) continue;
        float m = val(0);
#pragma unroll
        for (int i = 1; i < 127; i += 2) m = fmaxf(fmaxf(m, val(i)), val(i + 1));
        m = fmaxf(m, val(127));
        const float mm = m == -INFINITY ? 0.f : m;
        const F2 neg = pack2(-mm, -mm), cc = pack2(c1, c1);
        F2 s2 = pack2(0.f, 0.f), u2 = s2;
        if (a.part_u == nullptr) {
#pragma unroll
          for (int i = 0; i < 128; i += 2) {
            const float2 f = unpack2(mul2(add2(pack2(val(i), val(i + 1)), neg), cc));
            s2 = add2(s2, pack2(ex2(f.x), ex2(f.y)));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 128; i += 2) {
            const F2 d = mul2(add2(pack2(val(i), val(i + 1)), neg), cc);
            const float2 f = unpack2(d);
            const F2 e = pack2(ex2(f.x), ex2(f.y));
            s2 = add2(s2, e);
            u2 = fma2(e, d, u2);
          }
          const float2 w = unpack2(u2);
          if (!(fabsf(w.x + w.y) < INFINITY)) {
            // a logit of -inf among them: its 0 times -inf is left out (2^-1000 is 0 too)
            u2 = pack2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 128; ++i) {
              const float f = (val(i) - mm) * c1;
              u2 = fma2(pack2(ex2(f), 0.f), pack2(fmaxf(f, -1000.f), 0.f), u2);
            }
          }
        }
        if (row < n_rows) {
          const float2 s = unpack2(s2), w = unpack2(u2);
          const int64_t at = (int64_t)(u.n * (kBN / kPart) + half) * a.pitch + row;
          a.part_m[at] = m;
          a.part_s[at] = s.x + s.y;
          if (a.part_u != nullptr) a.part_u[at] = w.x + w.y;
          if (rel >= 0 && rel < live) {
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (i == rel) y = val(i);
            a.target_logit[row] = y;
          }
        }
      } else if constexpr (kMode == kGrad) {
        const bool on = row < n_rows;
        RowGrad g{0.f, 0.f, 0.f, 0.f};
        int rel = -1;
        if (on) {
          g = a.rows[row];
          rel = a.row_target[row] - a.v0 - col0;
        }
        const int live = a.width - col0;
        if (row0 < (n_rows + 63) / 64 * 64 && (a.low == 0 || row < a.low)) {   // the rows that the products read
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t (&x)[32] = v[c];
            auto val = [&](int i) { return __uint_as_float(x[i]); };
            const F2 cc = pack2(a.scale, a.scale), ll = pack2(-g.lse, -g.lse), to2 = pack2(kLog2e, kLog2e);
            const F2 aa = pack2(g.a, g.a), bb = pack2(g.b, g.b);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 lt = unpack2(mul2(fma2(pack2(val(i), val(i + 1)), cc, ll), to2));
              const F2 p = pack2(ex2(lt.x), ex2(lt.y));
              // 2^-1000 is 0: the clamp changes no product, and keeps 0 away from b * inf
              const F2 w = a.entropy ? fma2(bb, pack2(fmaxf(lt.x, -1000.f), fmaxf(lt.y, -1000.f)), aa) : aa;
              const float2 d = unpack2(mul2(p, w));
              x[i] = __float_as_uint(d.x);
              x[i + 1] = __float_as_uint(d.y);
            }
            if ((unsigned)(rel - 32 * c) < 32u) {
              float y = 0.f;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i == rel - 32 * c) x[i] = __float_as_uint(y = val(i) + g.zy);
              if (a.left != nullptr) {
                const float high = unpack_16bit(pack_16bit(y, 0.f, a.f16), a.f16).x;
                a.left[row] = fabsf(high) < INFINITY ? y - high : 0.f;
              }
            }
            if (live < 32 * c + 32 || !on) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!on || i >= live - 32 * c) x[i] = 0;
            }
            uint16_t* dst = a.d_out + (int64_t)row * a.d_pitch + col0 + 32 * c;
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = pack_16bit(val(2 * i), val(2 * i + 1), a.f16);
            store32(dst, w);
            store32(dst + 16, w + 8);
            if (a.low > 0) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 high = unpack_16bit(w[i], a.f16);
                w[i] = pack_16bit(val(2 * i) - high.x, val(2 * i + 1) - high.y, a.f16);
              }
              dst += a.low * a.d_pitch;
              store32(dst, w);
              store32(dst + 16, w + 8);
            }
          }
        }
        __syncwarp();
      } else {
        // 32 columns at a time, the next ones on their way out of TMEM under the arithmetic
        // (the sums of d's second parts are rows of their own)
        const bool on = row < n_rows || (a.low > 0 && row >= a.low && row < a.low + n_rows);
        const float f = u.w && a.w_factor != nullptr ? *a.w_factor : 1.f;
        // the rows of this warp that somebody reads, the columns that there are
        const bool wanted = u.w ? a.v0 + row0 < a.V : row0 < a.low + n_rows;
        const int live = a.H - col0;
        // What the rounding of d left at these 32 tokens' own rows, times the rows: to the lanes that have them, in the
        // order of the rows (lanes are columns here).
        uint32_t fixed = 0;
        float* fix = a.fixes + ((int64_t)blockIdx.x * kEpiWarps + ew) * (32 * 128);
        // (the word is looked at when the first columns are out of TMEM)
        const bool marked = u.w && wanted && live > 0 && lane < a.mark_words;
        const uint32_t mark_at = (uint32_t)(a.v0 + row0) / 32 * a.mark_words + lane;
        uint32_t mark_word = 0;
        if (kLeft) asm volatile("ld.global.b32 %0, [%1];" : "=r"(mark_word) : "l"(a.marks + (marked ? mark_at : 0)) : "memory");
        auto fix_up = [&] {
          const bool moved = a.always_gathered || n_rows < a.T;
          const uint16_t* x = static_cast<const uint16_t*>(moved ? a.x_gathered : a.x_all) + col0 + 4 * lane;
          const int64_t ldx = moved ? a.x_gathered_ld : a.x_all_ld;
          const int first = a.v0 + row0;
          int at = -1;                                         // the token whose sum is in registers
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
          auto store = [&] {
            if (at >= 0 && 4 * lane < live) *reinterpret_cast<float4*>(fix + at * 128 + 4 * lane) = sum;
          };
          // a block's next rows, with all of their loads on their way at once
          auto add = [&](auto flight, int t0, int mark, float e, uint32_t& hits) {
            constexpr int kFlight = decltype(flight)::value;
            int h[kFlight];
            uint2 q[kFlight];
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
              h[k] = __ffs(hits) - 1;
              hits &= hits - 1;
              q[k] = h[k] >= 0 && 4 * lane < live ? *reinterpret_cast<const uint2*>(x + (t0 + h[k]) * ldx) : make_uint2(0u, 0u);
            }
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
              if (h[k] < 0) break;
              const int to = __shfl_sync(0xFFFFFFFFu, mark, h[k]);
              const float f = __shfl_sync(0xFFFFFFFFu, e, h[k]);
              if (to != at) {
                store();
                at = to;
                sum = fixed >> to & 1u && 4 * lane < live ? *reinterpret_cast<const float4*>(fix + to * 128 + 4 * lane)
                                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                fixed |= 1u << to;
              }
              const float2 lo = unpack_16bit(q[k].x, a.f16), hi = unpack_16bit(q[k].y, a.f16);
              sum = make_float4(fmaf(f, lo.x, sum.x), fmaf(f, lo.y, sum.y), fmaf(f, hi.x, sum.z), fmaf(f, hi.y, sum.w));
            }
          };
          for (int w0 = 0; w0 < a.mark_words; w0 += 32) {
            const uint32_t mine = w0 == 0 ? mark_word : w0 + lane < a.mark_words ? a.marks[mark_at + w0] : 0u;
            for (uint32_t words = __ballot_sync(0xFFFFFFFFu, mine != 0); words != 0; words &= words - 1) {
              const int word = __ffs(words) - 1;
              for (uint32_t bits = __shfl_sync(0xFFFFFFFFu, mine, word); bits != 0; bits &= bits - 1) {
                const int t0 = ((w0 + word) * 32 + __ffs(bits) - 1) * 32;
                const int mark = t0 + lane < n_rows ? a.row_target[t0 + lane] - first : -1;
                const float e = t0 + lane < n_rows ? a.left[t0 + lane] : 0.f;
                uint32_t hits = __ballot_sync(0xFFFFFFFFu, (unsigned)mark < 32u);
                while (hits != 0) {
                  if (__popc(hits) > 4) add(std::integral_constant<int, 16>(), t0, mark, e, hits);
                  else add(std::integral_constant<int, 4>(), t0, mark, e, hits);
                }
              }
            }
          }
          store();
          __syncwarp();
        };
        // A stretch's columns, the next ones on their way.  (Two copies: where there are few rows few warps have a target
        // among their tokens.)
        uint32_t packed[32];
        auto columns = [&](auto fix_here, uint32_t taddr, uint32_t acc, int i, bool last) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t (&x)[32] = v[c & 1];
            if (c < 3) tmem_ld_32x32b_x32(taddr + 32 * (c + 1), v[(c + 1) & 1]);
            auto val = [&](int i) { return __uint_as_float(x[i]); };
            if (kMany && wanted && u.turns > 1) {
              float* part = a.long_sums + ((int64_t)blockIdx.x * kEpiWarps + ew) * (128 * 32) + (c * 128 + lane) * 8;
#pragma unroll
              for (int j = 0; j < 4; ++j) {   // 8 columns, a warp's 32 rows side by side
                if (i > 0) {
                  uint32_t o[8];
                  load32(part + j * 256, o);
#pragma unroll
                  for (int h = 0; h < 8; ++h) x[8 * j + h] = __float_as_uint(__uint_as_float(o[h]) + val(8 * j + h));
                }
                if (!last) store32(part + j * 256, x + 8 * j);
              }
            }
            if (!last) {
            } else if (!u.w) {
              if (wanted && on) {
                // float32 sums of dhidden, 8 columns at a time: this thread's alone
                float* dst = a.x_sums + ((int64_t)u.split * a.x_pitch + row) * a.H + col0 + 32 * c;
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                  if (32 * c + i >= live) break;
                  if (u.k0 >= u.k1) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[i + j] = 0;
                  }
                  if (!a.x_first) {
                    uint32_t o[8];
                    load32(dst + i, o);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[i + j] = __float_as_uint(__uint_as_float(o[j]) + val(i + j));
                  }
                  store32(dst + i, x + i);
                }
              }
            } else if (wanted && 64 * (c / 2) < live) {
              if (decltype(fix_here)::value && (fixed >> lane & 1u)) {
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  if (32 * c + i >= live) break;
                  const float4 o = *reinterpret_cast<const float4*>(fix + lane * 128 + 32 * c + i);
                  x[i] = __float_as_uint(val(i) + o.x), x[i + 1] = __float_as_uint(val(i + 1) + o.y);
                  x[i + 2] = __float_as_uint(val(i + 2) + o.z), x[i + 3] = __float_as_uint(val(i + 3) + o.w);
                }
              }
              // 64 columns of dweight's rows through a box: whole lines (rows behind V, columns behind H are cut)
#pragma unroll
              for (int i = 0; i < 16; ++i)
                packed[16 * (c & 1) + i] =
                    u.k0 >= u.k1 ? 0 : pack_16bit(val(2 * i) * f, val(2 * i + 1) * f, a.f16);
              if (c & 1) {
                if (lane == 0) bulk_wait_read<0>();
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  *reinterpret_cast<uint4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                      make_uint4(packed[4 * j], packed[4 * j + 1], packed[4 * j + 2], packed[4 * j + 3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                  tma_store_2d(&dweight, buf, col0 + 32 * (c - 1), a.v0 + row0);
                  bulk_commit();
                }
              }
            }
            tmem_ld_wait();
            tmem_loaded(v[(c + 1) & 1]);
            if (c == 2) release(acc);   // the last columns are in registers
          }
        };
        bool ready = true;
        for (int i = 0; i < (kMany ? u.turns : 1); ++i) {
          const bool last = !kMany || i + 1 == u.turns;
          const uint32_t acc = 2 * group + (turn & 1);
          if (!__all_sync(0xFFFFFFFFu, wait(&sm.accf[acc], (turn >> 1) & 1))) {
            ready = false;
            break;
          }
          ++turn;
          tc_fence_after();
          const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + acc * kBN + half * 128;
          tmem_ld_32x32b_x32(taddr, v[0]);
          tmem_ld_wait();
          tmem_loaded(v[0]);
          if (kLeft && i == 0) {
            if (!marked) mark_word = 0;
            if (__any_sync(0xFFFFFFFFu, mark_word != 0) || (a.mark_words > 32 && u.w && wanted && live > 0)) fix_up();
          }
          if (kLeft && last && fixed != 0) columns(std::true_type(), taddr, acc, i, last);
          else columns(std::false_type(), taddr, acc, i, last);
        }
        if (!ready) break;
      }
    }
    if (kMode == kProducts && lane == 0) bulk_wait_all<0>();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();   // no remote arrival or peer read is left in flight
  tc_fence_after();
  if (warp == 1) {
    if (kPair) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------------------ joining

struct JoinArgs {
  int64_t T, pitch;
  int parts, V;
  const float* m;
  const float* s;
  const float* u;
  const float* target_logit;
  const int32_t* targets;
  int32_t ignore;
  const int32_t* place;      // row -> gathered row or -1, nullable: itself
  const int32_t* n_rows;     // nullable
  float scale;
  float* logprob;
  float* lse;
  float* entropy;
  int* status;
};

// 32 rows a CTA, a lane each; warp w takes parts w, w + 32, ...
__global__ void __launch_bounds__(1024) head_join_kernel(const JoinArgs a) {
  __shared__ float sm_m[32][33], sm_s[32][33], sm_u[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_sync();
  const float c1 = a.scale * kLog2e;
  const int64_t t = (int64_t)blockIdx.x * 32 + lane;
  const int32_t y = t < a.T && a.targets != nullptr ? a.targets[t] : 0;
  const bool skip = t >= a.T || (a.targets != nullptr && y == a.ignore);
  const bool moved = a.n_rows != nullptr && *a.n_rows < a.T;
  const int64_t row = skip ? -1 : moved ? a.place[t] : t;
  float m = -INFINITY, s = 0.f, u = 0.f;
  auto join = [&](const float (&mi)[8], const float (&si)[8], const float (&ui)[8]) {   // s = 0: nothing allowed
    float top = m;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, mi[i]);
    // 2^-1000 is 0: the clamp changes no sum, and keeps 0 away from s * inf
    float d = s == 0.f ? 0.f : fmaxf((m - top) * c1, -1000.f), f = ex2(d);
    float s2 = f * s, u2 = f * fmaf(s, d, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d = si[i] == 0.f ? 0.f : fmaxf((mi[i] - top) * c1, -1000.f);
      f = ex2(d);
      s2 = fmaf(f, si[i], s2);
      u2 = fmaf(f, fmaf(si[i], d, ui[i]), u2);
    }
    m = top, s = s2, u = u2;
  };
  if (row >= 0) {
    for (int c0 = warp; c0 < a.parts; c0 += 32 * 8) {   // eight parts at a time
      float mi[8], si[8], ui[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + 32 * i;
        const int64_t at = c * a.pitch + row;
        const bool in = c < a.parts;
        mi[i] = in ? a.m[at] : -INFINITY;
        si[i] = in ? a.s[at] : 0.f;
        ui[i] = in && a.u != nullptr ? a.u[at] : 0.f;
      }
      join(mi, si, ui);
    }
  }
  sm_m[warp][lane] = m;
  sm_s[warp][lane] = s;
  sm_u[warp][lane] = u;
  __syncthreads();
  if (warp != 0 || t >= a.T) return;
  m = -INFINITY, s = 0.f, u = 0.f;
  for (int w = 0; w < 32; w += 8) {
    float mi[8], si[8], ui[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) mi[i] = sm_m[w + i][lane], si[i] = sm_s[w + i][lane], ui[i] = sm_u[w + i][lane];
    join(mi, si, ui);
  }
  if (skip) {
    if (a.logprob != nullptr) a.logprob[t] = 0.f;
    a.lse[t] = 0.f;
    if (a.entropy != nullptr) a.entropy[t] = 0.f;
    return;
  }
  const bool none = s == 0.f;                    // every token at -inf
  const float ln_s = logf(s);
  if (a.logprob != nullptr) {
    float lp = -INFINITY;
    if (y < 0 || y >= a.V) {
      set_status(a.status, kStatusBadInput);
      lp = NAN;
    } else if (!none) {
      lp = fmaf(a.target_logit[row] - m, a.scale, -ln_s);
    }
    a.logprob[t] = lp;
  }
  a.lse[t] = none ? -INFINITY : fmaf(m, a.scale, ln_s);
  if (a.entropy != nullptr) {
    const float h = ln_s - kLn2 * (u / s);
    a.entropy[t] = none || h < 0.f ? 0.f : h;    // round-off below 0
  }
}

// ------------------------------------------------------------------------------ gathering

// Gathered rows begin at whole lines (a 128-byte row of a box is one request of L2's then, not two).
__host__ __device__ inline int64_t row_pitch(int64_t H) { return (H + 63) / 64 * 64; }

struct GatherArgs {
  const void* hidden;
  int64_t ldh, T;
  int H, V, f16;
  const int32_t* targets;    // nullable
  int32_t ignore;
  float scale;
  const float* lse;          // nullable: forward
  const float* entropy;
  const float* dlogprob;
  const float* dentropy;
  int32_t* place;            // [T]
  int32_t* index;            // [T]
  int32_t* n_rows;
  float* factors;            // [0]: dweight's factor (half precision)
  float* row_factor;         // [rows]: dhidden's factors
  void* gathered;            // [rows rounded up to 64][row_pitch(H)], where not all rows take part
  int low;                   // where d has two parts: the copies' repetition
  void* weighted;            // the same times r / max r (half precision) and repeated (two parts), where either is so
  RowGrad* rows;
  int32_t* row_target;
  float* left;               // nullable, with marks: both cleared here, the marks set
  uint32_t* marks;
  int mark_words;
};

// Half precision holds d only down to 2^-24: a row travels as d / r with r a power of two above its
// weight, and its hidden row as hidden r / max r.  A row lighter than the heaviest has r up to 2^8 times its weight, so
// that its hidden row keeps its bits: d reaches 2^-30 of the weight there (an even share of 2^20 tokens is still a
// normal number), and the hidden row is as it is down to weights of 2^-8 of the heaviest, its numbers of 1 and more normal
// ones down to 2^-22.  Below that it loses a bit for each power of two; the result reaches 2^-30 of its own largest.
constexpr float kUp = 16384.f;    // d / r is below 1: 2^14 leaves room below the largest value
constexpr float kDown = 256.f;
__device__ __forceinline__ float row_weight(const GatherArgs& a, int64_t t) {
  const float g = a.dlogprob != nullptr ? fabsf(a.dlogprob[t]) : 0.f;
  const float h = a.dentropy != nullptr ? fabsf(a.dentropy[t]) : 0.f;
  const float w = a.scale * (g + 16.f * h);     // |p (ln p + entropy)| < 16
  if (!(w < INFINITY)) return 1.f;
  int e;
  frexpf(w, &e);
  return w == 0.f ? 0.f : ldexpf(1.f, min(max(e, -100), 100));
}

// The rows that take part, in their order: one CTA.
__global__ void __launch_bounds__(1024) head_select_kernel(const GatherArgs a) {
  __shared__ int sm_n[32];
  __shared__ float sm_r[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_sync();
  if (a.marks != nullptr) {
    const int64_t words = ((int64_t)a.V + 31) / 32 * a.mark_words;
    for (int64_t i = threadIdx.x; i < words; i += 1024) a.marks[i] = 0u;
  }
  constexpr int kEach = 8;   // rows a thread, one behind the other
  int base = 0;
  float r = 0.f;
  for (int64_t t0 = 0; t0 < a.T; t0 += 1024 * kEach) {
    const int64_t t1 = t0 + threadIdx.x * kEach;
    int32_t y[kEach];
    float lse[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const bool in = t1 + i < a.T;
      y[i] = in && a.targets != nullptr ? a.targets[t1 + i] : 0;
      lse[i] = in && a.lse != nullptr ? a.lse[t1 + i] : 0.f;
    }
    uint32_t on = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (t1 + i < a.T && (a.targets == nullptr || y[i] != a.ignore) && !(lse[i] < kLowestLse)) on |= 1u << i;
    int sum = __popc(on);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += o;
    }
    if (lane == 31) sm_n[warp] = sum;
    __syncthreads();
    int below = sm_n[lane], all = below;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, all, d);
      if (lane >= d) all += o;
    }
    int at = base + __shfl_sync(0xFFFFFFFFu, all - below, warp) + sum - __popc(on);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int64_t t = t1 + i;
      if (t < a.T) a.place[t] = (on >> i) & 1u ? at : -1;
      if ((on >> i) & 1u) {
        a.index[at++] = (int32_t)t;
        if (a.f16 && a.lse != nullptr) r = fmaxf(r, row_weight(a, t));
      }
    }
    base += __shfl_sync(0xFFFFFFFFu, all, 31);
    __syncthreads();
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) r = fmaxf(r, __shfl_xor_sync(0xFFFFFFFFu, r, d));
  if (lane == 0) sm_r[warp] = r;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 0; w < 32; ++w) r = fmaxf(r, sm_r[w]);
    *a.n_rows = base;
    if (a.factors != nullptr) {
      a.factors[0] = a.f16 ? r / kUp : 1.f;
      a.factors[1] = r;
    }
  }
}

// A warp a row: the gathered rows (zeros up to a multiple of 64), and what the gradient needs of them.
__global__ void __launch_bounds__(256) head_gather_kernel(const GatherArgs a) {
  grid_dep_sync();
  const int n = *a.n_rows;
  const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const bool scaled = a.f16 && a.lse != nullptr;
  if (i >= (n + 63) / 64 * 64) return;
  const int64_t t = i < n ? a.index[i] : 0;
  float ratio = 1.f;
  if (i < n && a.lse != nullptr) {
    const float r = scaled ? fminf(kDown * row_weight(a, t), a.factors[1]) : 1.f;
    if (scaled) ratio = a.factors[1] > 0.f ? r / a.factors[1] : 1.f;
    if (lane == 0) {
      const float up = !scaled ? 1.f : r > 0.f ? kUp / r : 0.f;
      const int32_t y = a.targets != nullptr ? a.targets[t] : -1;
      const bool hit = y >= 0 && y < a.V;   // a target that the forward refused adds nothing
      const float g = a.dlogprob != nullptr && hit ? a.dlogprob[t] * up : 0.f;
      const float h = a.dentropy != nullptr ? a.dentropy[t] * up : 0.f;
      RowGrad w;
      w.a = -a.scale * (g + (a.dentropy != nullptr ? h * a.entropy[t] : 0.f));
      w.b = -a.scale * h * kLn2;
      w.lse = a.lse[t];
      w.zy = a.scale * g;
      a.rows[i] = w;
      a.row_target[i] = hit ? y : -1;
      if (a.left != nullptr) {
        a.left[i] = 0.f;
        if (hit) atomicOr(&a.marks[(int64_t)(y / 32) * a.mark_words + i / 1024], 1u << (i / 32 % 32));
      }
      a.row_factor[i] = scaled ? r / kUp : 1.f;
    }
  }
  const int64_t pitch = row_pitch(a.H);
  const bool gather = n < a.T, copy = scaled || a.low > 0;   // else the rows are read where they are
  if (!gather && !copy) return;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.hidden) + t * a.ldh);
  for (int c0 = lane; c0 < a.H / 8; c0 += 32 * 8) {   // eight loads on their way
    uint4 q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) q[k] = i < n && c0 + 32 * k < a.H / 8 ? src[c0 + 32 * k] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = c0 + 32 * k;
      if (c >= a.H / 8) break;
      if (gather) reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.gathered) + i * pitch)[c] = q[k];
      if (scaled) {
        __half2* h = reinterpret_cast<__half2*>(&q[k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = __half22float2(h[j]);
          h[j] = __floats2half2_rn(f.x * ratio, f.y * ratio);
        }
      }
      if (copy && (a.low == 0 || i < a.low)) {
        uint16_t* dst = static_cast<uint16_t*>(a.weighted) + i * pitch;
        reinterpret_cast<uint4*>(dst)[c] = q[k];
        if (a.low > 0) reinterpret_cast<uint4*>(dst + a.low * pitch)[c] = q[k];
      }
    }
  }
}

struct FinishArgs {
  int64_t T, pitch;
  int H, f16, splits, low;
  const int32_t* place;
  const float* row_factor;
  const float* sums;         // [splits][pitch][H]
  const float* left;         // nullable: d has two parts
  const int32_t* row_target;
  const void* weight;
  int64_t ldw;
  void* out;
};

__global__ void __launch_bounds__(256) head_finish_kernel(const FinishArgs a) {
  grid_dep_sync();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = a.H / 8;
  const int64_t t = i / per;
  if (t >= a.T) return;
  const int c = (int)(i - t * per) * 8;
  const int place = a.place[t];
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (place >= 0) {
    // the sums of d's second parts first, where there are some; eight loads on their way
    const int all = a.low > 0 ? 2 * a.splits : a.splits;
    for (int i0 = 0; i0 < all; i0 += 8) {
      float4 x[8][2];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + j, split = i < a.splits ? i : i - a.splits;
        const int64_t row = split * a.pitch + (a.low > 0 && i < a.splits ? a.low : 0) + place;
        const float4* p = reinterpret_cast<const float4*>(a.sums + row * a.H + c);
        x[j][0] = i < all ? p[0] : make_float4(0.f, 0.f, 0.f, 0.f);
        x[j][1] = i < all ? p[1] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[0] += x[j][0].x, v[1] += x[j][0].y, v[2] += x[j][0].z, v[3] += x[j][0].w;
        v[4] += x[j][1].x, v[5] += x[j][1].y, v[6] += x[j][1].z, v[7] += x[j][1].w;
      }
    }
    const float f = a.row_factor[place], e = a.left != nullptr ? a.left[place] : 0.f;
    if (e != 0.f) {   // what the rounding of the target's d left
      const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.weight) +
                                                      a.row_target[place] * a.ldw + c);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = unpack_16bit(w[j], a.f16);
        v[2 * j] = fmaf(e, x.x, v[2 * j]), v[2 * j + 1] = fmaf(e, x.y, v[2 * j + 1]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= f;
  }
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (a.f16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + t * a.H + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

// ------------------------------------------------------------------------------ host

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// Up to a tile's 128 rows by single CTAs, more by pairs.  131072 x 2048, forward / backward (one number a d): 128 rows
// 100 / 300 us against 106 / 366 by pairs, 200 rows 107 / 385 us against 139 / 423 by single CTAs.
bool pairs(int64_t T) { return T > kBM; }

struct ForwardPlan {
  int64_t pitch;
  int parts;
  bool gather;
  size_t place, index, n, target, gathered, m, s, u, total;
};
ForwardPlan forward_plan(int64_t T, int64_t V, int64_t H) {
  ForwardPlan p;
  p.pitch = round_up(T, 32);
  p.parts = (int)((V + kPart - 1) / kPart);
  // Fewer rows are one row of tiles whatever takes part: 256 of them take 107 us, 112 with the two launches; 512 rows
  // 175 us against 170 without them, and with every other row ignored 113 against 171.
  p.gather = T > 2 * kBM;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) & ~size_t(255);
    return o;
  };
  p.n = take(4);
  p.place = take(4 * (size_t)T);
  p.index = take(4 * (size_t)T);
  p.target = take(4 * (size_t)p.pitch);
  p.gathered = take(p.gather ? 2 * (size_t)round_up(T, 64) * (size_t)row_pitch(H) : 0);
  p.m = take(4 * (size_t)p.parts * (size_t)p.pitch);
  p.s = take(4 * (size_t)p.parts * (size_t)p.pitch);
  p.u = take(4 * (size_t)p.parts * (size_t)p.pitch);
  p.total = at;
  return p;
}

struct BackwardPlan {
  int64_t rows;              // of d and of the sums: T rounded up to 64, or twice `low`
  int low;                   // where d has two parts, T rounded up to 16; else 0
  int64_t piece;             // columns of a piece of the vocabulary
  int splits;
  bool many;
  int mark_words;
  size_t n, factors, place, index, grad, target, row_factor, gathered, weighted, d, sums, long_sums, left, marks, fixes,
      total;
};
BackwardPlan backward_plan(int64_t T, int64_t V, int64_t H) {
  BackwardPlan p;
  p.low = T <= kTwoParts ? (int)round_up(T, 16) : 0;
  p.rows = p.low > 0 ? 2 * p.low : round_up(T, 64);
  // Pieces of 2^28 elements: 8192 x 131072 x 2048 8.06 ms with all rows, of 2^27 8.34, of 2^29 (1 GB) 7.98.
  const int64_t vp = round_up(V, 256);
  int64_t piece = std::max<int64_t>(8192, round_up(((int64_t)1 << 28) / p.rows, 256));
  const int64_t pieces = (vp + piece - 1) / piece;
  p.piece = round_up((vp + pieces - 1) / pieces, 256);
  // Few rows: dhidden's contraction is cut so that every SM has a part of it, into 32 at most (48 x 131072 x 512:
  // 148 us; 16 163, 64 190).
  const int64_t tile = pairs(T) ? 2 * kBM : kBM, tiles = (T + tile - 1) / tile * ((H + 255) / 256);
  p.splits = pieces == 1 ? (int)std::min<int64_t>(std::max<int64_t>(1, (pairs(T) ? kMaxCtas / 2 : kMaxCtas) / tiles), 32) : 1;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) & ~size_t(255);
    return o;
  };
  p.n = take(4);
  p.factors = take(8);
  p.place = take(4 * (size_t)T);
  p.index = take(4 * (size_t)T);
  p.grad = take(sizeof(RowGrad) * (size_t)T);
  p.target = take(4 * (size_t)T);
  p.row_factor = take(4 * (size_t)T);
  // The areas are as large as any smaller T needs them, so that a workspace for the largest batch serves the others:
  // rows <= `most`; a piece is at most 2^28 / rows + 256 or 8192 columns; splits are at most 32, and their tiles at most
  // one for each CTA (of 128 rows, or 256 a pair), or there is one split.
  const int64_t most = p.low > 0 && T <= 32 ? p.rows : std::max<int64_t>(round_up(T, 64), 128);
  const int64_t cells = std::min(most * vp, std::max(((int64_t)1 << 28) + 256 * most, 8192 * most));
  const int64_t sums = std::max(most, std::min(32 * most, kMaxCtas * kBM / ((H + 255) / 256)));
  p.gathered = take(2 * (size_t)most * (size_t)row_pitch(H));
  p.weighted = take(2 * (size_t)most * (size_t)row_pitch(H));   // (a call does not say whether it is half precision)
  p.d = take(2 * (size_t)cells);
  p.sums = take(4 * (size_t)sums * (size_t)H);
  // a contraction of dhidden is at most V long, of dweight T; `many`: one of them is longer than a stretch
  p.long_sums = take(std::max(T, V) > kLong * kBK ? kMaxCtas * kLongBytes : 0);
  const int64_t x_blocks = (std::min(p.piece, V) + kBK - 1) / kBK;
  p.many = (x_blocks + p.splits - 1) / p.splits > kLong || T > kLong * kBK;
  p.mark_words = (int)((T + 1023) / 1024);
  p.left = take(4 * (size_t)T);
  p.marks = take(4 * (size_t)((V + 31) / 32) * (size_t)p.mark_words);
  p.fixes = take(p.low > 0 ? 0 : kMaxCtas * kLongBytes);
  p.total = at + 240;        // the areas begin at the first whole 256 bytes of a 16-byte aligned workspace
  return p;
}

template <int kMode, bool kPair, bool kMany, bool kLeft>
cudaError_t launch_head(const CUtensorMap (&maps)[5], const HeadArgs& a, int64_t units, cudaStream_t s) {
  const auto fn = head_kernel<kMode, kPair, kMany, kLeft>;
  static std::atomic<bool> attr_set[64];
  cudaError_t err = set_smem_attr_once(attr_set, (const void*)fn, (int)smem_bytes<kMode, kPair>());
  if (err != cudaSuccess || units == 0) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kPair ? 2 : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes<kMode, kPair>();
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = kPair ? 2 : 1;
  int64_t clusters = kPair ? num_sms() / 2 : num_sms();
  clusters = std::min<int64_t>({clusters, units, kMaxCtas / (kPair ? 2 : 1)});
  cfg.gridDim = dim3((unsigned)(clusters * (kPair ? 2 : 1)), 1, 1);
  return cudaLaunchKernelEx(&cfg, fn, maps[0], maps[1], maps[2], maps[3], maps[4], a);
}
template <int kMode>
cudaError_t launch_head(bool pair, const CUtensorMap (&maps)[5], const HeadArgs& a, int64_t units, cudaStream_t s) {
  if constexpr (kMode == kProducts) {   // (pairs have more than 64 rows, and one number a d)
    const bool many = a.long_sums != nullptr;
    if (pair) return many ? launch_head<kMode, true, true, true>(maps, a, units, s) : launch_head<kMode, true, false, true>(maps, a, units, s);
    if (a.left != nullptr)
      return many ? launch_head<kMode, false, true, true>(maps, a, units, s) : launch_head<kMode, false, false, true>(maps, a, units, s);
    return many ? launch_head<kMode, false, true, false>(maps, a, units, s) : launch_head<kMode, false, false, false>(maps, a, units, s);
  } else {
    return pair ? launch_head<kMode, true, false, false>(maps, a, units, s) : launch_head<kMode, false, false, false>(maps, a, units, s);
  }
}

}  // namespace

size_t head_workspace(int64_t T, int64_t V, int64_t H, bool backward) {
  return backward ? backward_plan(T, V, H).total : forward_plan(T, V, H).total;
}

cudaError_t launch_head_logprobs(const void* hidden, int64_t ldh, const void* weight, int64_t ldw, int dtype, int64_t T,
                                 int64_t V, int64_t H, const int32_t* targets, int32_t ignore, float scale,
                                 float* logprob, float* lse, float* entropy, void* workspace, cudaStream_t s) {
  const ForwardPlan p = forward_plan(T, V, H);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto f32 = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  auto i32 = [&](size_t o) { return reinterpret_cast<int32_t*>(ws + o); };
  const bool gather = p.gather && targets != nullptr, pair = pairs(T);
  const int x_rows = (int)std::min<int64_t>(64, round_up(T, 8));
  const CUtensorMapDataType dt = dtype == kActF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap maps[5];
  if (!make_tensor_map(&maps[0], hidden, T, H, 2 * ldh, x_rows, dt, 2) ||
      !make_tensor_map(&maps[2], weight, V, H, 2 * ldw, 64, dt, 2))
    return cudaErrorInvalidValue;
  maps[1] = maps[0];
  if (gather && !make_tensor_map(&maps[1], ws + p.gathered, round_up(T, 64), H, 2 * row_pitch(H), 64, dt, 2))
    return cudaErrorInvalidValue;
  maps[3] = maps[4] = maps[2];
  cudaError_t err = cudaSuccess;
  if (gather) {
    GatherArgs g{};
    g.hidden = hidden, g.ldh = ldh, g.T = T, g.H = (int)H, g.V = (int)V, g.f16 = dtype == kActF16;
    g.targets = targets, g.ignore = ignore;
    g.place = i32(p.place), g.index = i32(p.index), g.n_rows = i32(p.n), g.gathered = ws + p.gathered;
    err = launch_pdl(false, head_select_kernel, dim3(1), dim3(1024), 0, s, g);
    if (err == cudaSuccess)
      err = launch_pdl(true, head_gather_kernel, dim3((unsigned)(round_up(T, 64) / 8)), dim3(256), 0, s, g);
    if (err != cudaSuccess) return err;
  }
  HeadArgs a{};
  a.T = T, a.x_rows = x_rows, a.n_rows = gather ? i32(p.n) : nullptr, a.V = (int)V, a.H = (int)H, a.f16 = dtype == kActF16;
  a.scale = scale, a.status = device_status_ptr();
  a.targets = targets, a.index = gather ? i32(p.index) : nullptr;
  a.part_m = f32(p.m), a.part_s = f32(p.s), a.part_u = entropy != nullptr ? f32(p.u) : nullptr, a.pitch = p.pitch;
  a.target_logit = f32(p.target), a.width = (int)V;
  const int64_t tile = pair ? 2 * kBM : kBM;
  const int64_t cols = tile_cols(kStats, pair);
  err = launch_head<kStats>(pair, maps, a, (T + tile - 1) / tile * ((V + cols - 1) / cols), s);
  if (err != cudaSuccess) return err;
  JoinArgs j{T, p.pitch, p.parts, (int)V, a.part_m, a.part_s, a.part_u, a.target_logit, targets, ignore,
             gather ? i32(p.place) : nullptr, a.n_rows, scale, logprob, lse, entropy, a.status};
  return launch_pdl(true, head_join_kernel, dim3((unsigned)((T + 31) / 32)), dim3(1024), 0, s, j);
}

cudaError_t launch_head_logprobs_backward(const void* hidden, int64_t ldh, const void* weight, int64_t ldw, int dtype,
                                          int64_t T, int64_t V, int64_t H, const int32_t* targets, int32_t ignore,
                                          float scale, const float* lse, const float* entropy, const float* dlogprob,
                                          const float* dentropy, void* dhidden, void* dweight, void* workspace,
                                          cudaStream_t s) {
  const BackwardPlan p = backward_plan(T, V, H);
  // d and the float32 sums are accessed 32 bytes at a time
  uint8_t* ws = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~uintptr_t(255));
  auto f32 = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  auto i32 = [&](size_t o) { return reinterpret_cast<int32_t*>(ws + o); };
  const bool f16 = dtype == kActF16, pair = pairs(T);
  const CUtensorMapDataType dt = f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  GatherArgs g{};
  g.hidden = hidden, g.ldh = ldh, g.T = T, g.H = (int)H, g.V = (int)V, g.f16 = f16;
  g.targets = targets, g.ignore = ignore, g.scale = scale;
  g.lse = lse, g.entropy = entropy, g.dlogprob = dlogprob, g.dentropy = dentropy;
  g.place = i32(p.place), g.index = i32(p.index), g.n_rows = i32(p.n), g.factors = f32(p.factors);
  g.row_factor = f32(p.row_factor), g.gathered = ws + p.gathered, g.weighted = ws + p.weighted;
  if (p.low == 0)
    g.left = f32(p.left), g.marks = reinterpret_cast<uint32_t*>(ws + p.marks), g.mark_words = p.mark_words;
  g.low = p.low, g.rows = reinterpret_cast<RowGrad*>(ws + p.grad), g.row_target = i32(p.target);
  cudaError_t err = launch_pdl(false, head_select_kernel, dim3(1), dim3(1024), 0, s, g);
  if (err == cudaSuccess)
    err = launch_pdl(true, head_gather_kernel, dim3((unsigned)(round_up(T, 64) / 8)), dim3(256), 0, s, g);
  if (err != cudaSuccess) return err;

  HeadArgs a{};
  const int x_rows = (int)std::min<int64_t>(64, round_up(T, 8));
  a.T = T, a.x_rows = x_rows, a.n_rows = i32(p.n), a.V = (int)V, a.H = (int)H, a.f16 = f16;
  a.scale = scale, a.status = device_status_ptr();
  a.low = p.low;
  const bool weighted = f16 || p.low > 0;   // the rows that dweight's product reads are copies
  a.rows = g.rows, a.row_target = g.row_target, a.entropy = dentropy != nullptr, 
  a.d_out = reinterpret_cast<uint16_t*>(ws + p.d), a.d_pitch = p.piece, a.x_sums = f32(p.sums);
  a.long_sums = p.many ? f32(p.long_sums) : nullptr;
  a.x_splits = p.splits, a.x_pitch = p.rows;
  a.left = g.left, a.marks = g.marks, a.mark_words = g.mark_words, a.fixes = f32(p.fixes);
  a.x_all = hidden, a.x_all_ld = ldh, a.x_gathered = weighted ? g.weighted : g.gathered, a.x_gathered_ld = row_pitch(H);
  a.want_x = dhidden != nullptr, a.want_w = dweight != nullptr;
  a.w_factor = f16 ? g.factors : nullptr;
  CUtensorMap grad[5], prod[5];
  if (!make_tensor_map(&grad[0], hidden, T, H, 2 * ldh, x_rows, dt, 2) ||
      !make_tensor_map(&grad[1], ws + p.gathered, round_up(T, 64), H, 2 * row_pitch(H), x_rows, dt, 2) ||
      !make_tensor_map(&grad[2], weight, V, H, 2 * ldw, 64, dt, 2) ||
      !make_tensor_map(&grad[3], ws + p.d, p.rows, p.piece, 2 * p.piece, 64, dt, 2))
    return cudaErrorInvalidValue;
  prod[2] = grad[2], prod[3] = grad[3], prod[4] = grad[4] = grad[3];
  if (dweight != nullptr && !make_tensor_map(&prod[4], dweight, V, H, 2 * H, 32, dt, 2)) return cudaErrorInvalidValue;
  if (!make_tensor_map(&prod[0], hidden, T, H, 2 * ldh, 64, dt, 2) ||
      !make_tensor_map(&prod[1], ws + (weighted ? p.weighted : p.gathered), p.low > 0 ? p.rows : round_up(T, 64), H,
                       2 * row_pitch(H), 64, dt, 2))
    return cudaErrorInvalidValue;
  const int64_t tile = pair ? 2 * kBM : kBM, xn = (H + 255) / 256, cols = tile_cols(kGrad, pair);
  for (int64_t v0 = 0; v0 < V; v0 += p.piece) {
    a.v0 = (int)v0, a.width = (int)std::min<int64_t>(p.piece, V - v0), a.x_first = v0 == 0;
    a.always_gathered = false;
    err = launch_head<kGrad>(pair, grad, a, (T + tile - 1) / tile * ((a.width + cols - 1) / cols), s);
    if (err != cudaSuccess) return err;
    const int64_t units = (a.want_x ? (T + tile - 1) / tile * xn * p.splits : 0) +
                          (a.want_w ? (a.width + tile - 1) / tile * xn : 0);
    a.always_gathered = weighted;
    err = launch_head<kProducts>(pair, prod, a, units, s);
    if (err != cudaSuccess) return err;
  }
  if (dhidden == nullptr) return cudaSuccess;
  FinishArgs f{T, p.rows, (int)H, f16, p.splits, a.low, g.place, g.row_factor, f32(p.sums), g.left, g.row_target,
               weight, ldw, dhidden};
  return launch_pdl(true, head_finish_kernel, dim3((unsigned)((T * (H / 8) + 255) / 256)), dim3(256), 0, s, f);
}

}  // namespace nvfp4
