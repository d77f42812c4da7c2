// Distillation from a teacher's top logits: a row's loss over the student's logits z, and its
// gradient in the same call.
//
//   c = scale z, lse = ln sum exp(c), p = exp(c - lse);  S = the teacher's list, values t
//   tail off: q = softmax(t over S);   tail on: q = exp(t), q_r = max(0, 1 - sum q)
//   L = sum_S q (ln q - (c - lse))  [+ q_r (ln q_r - ln p_r), p_r = the student's mass outside S]
//   dL/dc = M p - q on S;  outside M p, or with the tail M p - q_r p / p_r = exp(c - lse_r) (M p_r - q_r)
//   M = the mass that L counts: 1, but with the tail sum q where that is above 1 or where no token outside
//   S is allowed (p_r = 0: nothing stands for the rest, and its term is left out of L)
//
// With the tail, the sum over the tokens outside S is taken on its own, with its own running
// maximum: 1 - sum_S p would cancel when the student's mass lies on S.  lse then is that of the
// two parts.  The gradient is 2^((z - m) scale log2 e) times one number of the row, and on S a
// value that is written over it afterwards.
// One warp of each CTA reduces the list to a few sums while the row arrives; the row's maximum
// enters them afterwards, so nothing but scalars follows the exchange between CTAs.
//
// The loss alone streams like the log probabilities; a bitmap of S in shared memory leaves the
// listed tokens out (8192 x 131072 BF16, K = 64: 306 us with the tail, 317 without, 7.0 and 6.8 TB/s).  With the gradient a row's slices lie in the shared memory of a cluster
// between the sum and the gradient, so HBM sees the row read once and written once
// (8192 x 131072 BF16, K = 64 with the tail: 706 us, 6.1 TB/s, 90% of a copy's rate; 1000 x 50021
// float16, K = 100: 53 us, 3.8 TB/s).  What bounds it is the row's chain -- arrival, sum,
// exchange, gradient -- of which an SM has three to four under way: warps wait at a barrier 5 of
// 12 cycles, the issue slots are used to half.  Measured and not kept: the row read again from L2
// instead of staged (4096 rows: 600-660 us against 400), the gradient written into the stage and
// copied out in bulk (1008 us against 870 at that time), two stages where a slice is a CTA's
// alone (780 us).  A slice too long for the shared memory is read again.
#include "launch.h"
#include "ptx.cuh"
#include "status.cuh"
#include "vocab.cuh"

namespace nvfp4 {
namespace {

namespace cg = cooperative_groups;

struct DistillArgs {
  const void* logits;
  int64_t ld;
  int V;
  const int32_t* ids;
  const float* values;
  int K;
  float scale;
  const float* dloss;
  float *loss, *lse;
  void* dlogits;
  int64_t ldd;
  int* status;
};

// The list of a row, and its sums.  mz is the maximum of its logits, s = sum 2^((z - mz) c1),
// A = sum q ln q, B = scale sum q (z - mz), Q = sum q.
struct ListSmem {
  int id[kMaxList];   // of the K entries; the places up to a multiple of 32 hold -1
  float q[kMaxList], z[kMaxList];
  float mz, s, A, B, Q;
  int live, bad;
  int twice;   // one of the ids in this CTA's slices stands there twice
};
// What the row's sums give: outside the list the gradient is coef 2^((z - mb) c1); at a listed token
// M p = inv 2^((z - m) c1).  With the tail, st covers the tokens outside the list.
struct RowResult {
  float mb, coef, m, inv;
  float rest, total;   // 2^((mb - m) c1) and the sum over all tokens, both relative to m
};
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
struct DistillSmem {
  Stats part[kMaxSlices][kVocabWarps];
  int twice[kMaxSlices];   // by CTA
  ListSmem list;
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The listed tokens of a CTA's slices: a bit a token, ordered so that a thread's four chunks of a batch are
// one word: word (r / 1024) 256 + r % 256 of chunk r of a slice, byte r / 256 % 4 of it.
struct Marks {
  unsigned* words;
  int first, per, count;   // first chunk; chunks a slice; chunks in all
  static __host__ __device__ int slice_words(int per) { return (per + 1023) / 1024 * 256; }
  __device__ __forceinline__ bool has(int id) const { return id >= 8 * first && id < 8 * (first + count); }
  __device__ __forceinline__ unsigned* word(int id) const {
    const int c = (id >> 3) - first, s = c / per, r = c - s * per;
    return words + s * slice_words(per) + (r >> 10) * 256 + (r & 255);
  }
  __device__ __forceinline__ unsigned bit(int id) const {
    const int c = (id >> 3) - first, r = c % per;
    return 1u << (8 * ((r >> 8) & 3) + (id & 7));
  }
  // of the batch that begins r chunks into slice s of the CTA's
  __device__ __forceinline__ unsigned batch(int s, int r) const {
    return words[s * slice_words(per) + (r >> 10) * 256 + (r & 255)];
  }
};

// A warp's part of a row's list: entries lane + 32 j.  Read in two steps (the ids and values, then
// the logits at the ids), so that the steps' latencies can lie behind other work.
template <typename E, bool kTail>
struct ListRegs {
  static constexpr int N = kMaxList / 32;
  int id[N];
  float v[N], zi[N];
  bool bad = false, live = false;
  int used;          // entries a lane: ceil(K / 32)
  __device__ __forceinline__ void read(const DistillArgs& a, int64_t t) {
    used = (a.K + 31) >> 5;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j >= used) break;
      const int i = (threadIdx.x & 31) + 32 * j;
      id[j] = i < a.K ? a.ids[t * a.K + i] : -1;
      v[j] = i < a.K ? a.values[t * a.K + i] : -INFINITY;
    }
  }
  __device__ __forceinline__ void gather(const DistillArgs& a, const E* z) {
    bad = live = false;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j >= used) break;
      if (id[j] < 0 || id[j] >= a.V) {
        bad |= id[j] != -1;
        id[j] = -1;
        v[j] = -INFINITY;
      }
      zi[j] = id[j] >= 0 ? to_f32(z[id[j]]) : -INFINITY;
      live |= kTail ? id[j] >= 0 : !(v[j] == -INFINITY);   // NaN lives
    }
  }
  // Marks the ids that lie in the CTA's slices in `listed` (clear there) and leaves the sums in sm.
  template <bool kMark>
  __device__ __forceinline__ void reduce(float scale, const Marks& listed, ListSmem& sm) const {
    const float c1 = scale * kLog2e;
    const int lane = threadIdx.x & 31;
    bool again = false;
    float mv = -INFINITY, mz = -FLT_MAX;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j >= used) break;
      if (kMark && listed.has(id[j])) {
        const unsigned bit = listed.bit(id[j]);
        again |= (atomicOr(listed.word(id[j]), bit) & bit) != 0;
      }
      mv = fmaxf(mv, v[j]);
      mz = fmaxf(mz, zi[j]);
    }
    mz = warp_max(mz);
    if (!kTail) mv = warp_max(mv);
    float e[N], esum = 0.f, s = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j >= used) break;
      e[j] = id[j] >= 0 ? expf(kTail ? v[j] : v[j] - mv) : 0.f;
      esum += e[j];
      if (!(zi[j] == -INFINITY)) s += ex2((zi[j] - mz) * c1);
    }
    if (!kTail) esum = warp_sum(esum);
    const float ln_e = kTail ? 0.f : logf(esum);
    float A = 0.f, B = 0.f, Q = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j >= used) break;
      const float q = kTail ? e[j] : e[j] / esum;
      if (q != 0.f) {   // 0 ln 0 = 0
        A += q * (kTail ? v[j] : v[j] - mv - ln_e);
        // (q scale first: a difference of the lowest values' size times more than 1 is beyond float32)
        B += zi[j] == -INFINITY ? -INFINITY : q * scale * (zi[j] - mz);
      }
      Q += q;
      const int i = lane + 32 * j;
      sm.id[i] = id[j];
      sm.q[i] = q;
      sm.z[i] = zi[j];
    }
    s = warp_sum(s);
    A = warp_sum(A);
    B = warp_sum(B);
    Q = warp_sum(Q);
    const int any_bad = __any_sync(0xffffffffu, bad), any_live = __any_sync(0xffffffffu, live);
    const int any_twice = __any_sync(0xffffffffu, again);
    if (lane == 0) {
      sm.mz = mz;
      sm.s = s;
      sm.A = A;
      sm.B = B;
      sm.Q = Q;
      sm.bad = any_bad;
      sm.live = any_live;
      sm.twice = any_twice;
    }
  }
  // The same in a row that lies in shared memory: the listed tokens there become -inf (with the tail;
  // else they keep their values).  Returns whether an id stands there twice: each entry
  // first writes its number into its token's place.
  template <typename Stage>
  __device__ __forceinline__ bool take_out(const Stage& stage) const {
    bool again = false;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j >= used) break;
      if (stage.has(id[j])) *stage.word(id[j]) = static_cast<uint16_t>((threadIdx.x & 31) + 32 * j);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j >= used) break;
      if (stage.has(id[j])) again |= *stage.word(id[j]) != (threadIdx.x & 31) + 32 * j;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j >= used) break;
      if (stage.has(id[j])) store_one(reinterpret_cast<E*>(stage.at(id[j])), kTail ? -INFINITY : zi[j]);
    }
    __syncwarp();
    return __any_sync(0xffffffffu, again);
  }
  // Clears the marks that reduce() made for this list.
  __device__ __forceinline__ void clear(const ListSmem& sm, const Marks& listed) const {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j >= used) break;
      const int i = sm.id[(threadIdx.x & 31) + 32 * j];
      if (listed.has(i)) *listed.word(i) = 0;
    }
    __syncwarp();
  }
};

template <bool kTail>
__device__ __forceinline__ RowResult finish_row(const Stats& st, const ListSmem& l, float c1) {
  RowResult r;
  const float mass = !kTail ? 1.f : st.s == 0.f ? l.Q : fmaxf(1.f, l.Q);   // M
  r.mb = st.m;
  if (kTail) {
    r.m = fmaxf(l.mz, st.m);
    r.rest = ex2((st.m - r.m) * c1);
    r.total = fmaf(r.rest, st.s, l.s == 0.f ? 0.f : ex2((l.mz - r.m) * c1) * l.s);
    // (M p_r - q_r) / sum outside the list
    r.coef = st.s == 0.f ? 0.f : mass * r.rest * rcp(r.total) - fmaxf(0.f, 1.f - l.Q) * rcp(st.s);
  } else {
    r.m = st.m;
    r.rest = 1.f;
    r.total = st.s;
    r.coef = st.s == 0.f ? 0.f : rcp(st.s);
  }
  r.inv = r.total == 0.f ? 0.f : mass * rcp(r.total);
  return r;
}
struct RowLoss {
  float loss, lse;
};
template <bool kTail>
__device__ __forceinline__ RowLoss row_loss(const Stats& st, const RowResult& r, const ListSmem& l, float scale) {
  const float ln_s = logf(r.total);
  float tail = 0.f;
  if (kTail && st.s != 0.f) {   // some token outside the list is allowed (NaN counts)
    const float qr = fmaxf(0.f, 1.f - l.Q);
    // ln p_r = scale (mb - m) + ln s_r - ln s, each part times q_r
    if (qr > 0.f) tail = fmaf(-(qr * scale), r.mb - r.m, qr * (logf(qr) - (logf(st.s) - ln_s)));
  }
  // sum q (ln q - ln p) with ln p = scale (z - m) - ln s; a student without any allowed token
  // has p = 0 everywhere
  RowLoss o;
  if (l.Q == 0.f) o.loss = tail;
  else if (r.total == 0.f) o.loss = INFINITY;
  else o.loss = l.A - (l.B + l.Q * scale * (l.mz - r.m)) + ln_s * l.Q + tail;
  o.lse = r.total == 0.f ? -INFINITY : fmaf(r.m, scale, ln_s);
  return o;
}

// The gradient at entry j of the list: w (M p - q), 0 at an excluded token.
__device__ __forceinline__ float listed_gradient(const ListSmem& l, int j, const RowResult& r, float c1, float w) {
  const float z = l.z[j];
  return z == -INFINITY ? 0.f : w * (ex2((z - r.m) * c1) * r.inv - l.q[j]);
}

// The listed tokens of a batch become -inf.
template <typename E>
__device__ __forceinline__ void leave_out(Chunk<E> (&raw)[4], unsigned marks) {
  if (marks == 0) return;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (marks >> (8 * k) & 255u)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (marks >> (8 * k + i) & 1) raw[k].leave_out(i);
}

// The loss alone.
template <typename E, bool kTail>
__global__ void __launch_bounds__(kVocabThreads) distill_topk_kernel(const DistillArgs a) {
  extern __shared__ __align__(16) unsigned listed_words[];
  __shared__ DistillSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int64_t t = blockIdx.x / ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (ctas > 1) cluster.barrier_arrive();   // met below, before anything is written to another CTA
  const Row<E> row(static_cast<const E*>(a.logits), a.ld, t, a.V);
  const int slices = vocab_slices(a.V);
  const float c1 = a.scale * kLog2e;
  const int s0 = rank * (slices / ctas), s1 = s0 + slices / ctas;
  int first, end, unused;
  slice_range(a.V, slices, s0, first, unused);
  slice_range(a.V, slices, s1 - 1, unused, end);
  const int per = (((a.V + 7) >> 3) + slices - 1) / slices;
  const Marks listed{listed_words, first, per, end - first};
  for (int i = tid; i < (s1 - s0) * Marks::slice_words(per); i += kVocabThreads) listed_words[i] = 0;
  ListRegs<E, kTail> mine;
  if (warp == 0) {
    mine.read(a, t);
    mine.gather(a, row.p);
  }
  __syncthreads();
  if (warp == 0) mine.template reduce<true>(a.scale, listed, sm.list);
  __syncthreads();
  if (ctas > 1) cluster.barrier_wait();
  const ListSmem& l = sm.list;
  const bool dead = l.bad || !l.live;
  if (!dead)
    for (int s = s0; s < s1; ++s) {
      int f, e;
      slice_range(a.V, slices, s, f, e);
      Running<E, false> run;
      for_batches(row, f, e, [&](int c, Chunk<E>(&raw)[4], int left) {
        if (kTail) leave_out(raw, listed.batch(s - s0, c - f));
        run.add(raw, left, c1);
      });
      const Stats st = run.warp(c1);
      if (lane == 0) *(ctas == 1 ? &sm.part[s][warp] : cluster.map_shared_rank(&sm.part[s][warp], 0)) = st;
    }
  if (ctas > 1) {
    if (tid == 0) *cluster.map_shared_rank(&sm.twice[rank], 0) = l.twice;
    cluster.sync();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }
  if (warp != 0) return;
  bool bad = l.bad || (ctas == 1 && l.twice);
  for (int r = 0; ctas > 1 && r < ctas; ++r) bad |= sm.twice[r] != 0;
  RowLoss o{0.f, 0.f};
  if (!dead) {
    const Stats st = Running<E, false>::join_slices(sm.part, slices, c1);
    o = row_loss<kTail>(st, finish_row<kTail>(st, l, c1), l, a.scale);
  }
  if (lane == 0) {
    if (bad) set_status(a.status, kStatusBadInput);
    a.loss[t] = bad ? NAN : o.loss;
    if (a.lse != nullptr) a.lse[t] = bad ? 0.f : o.lse;
  }
}

// A CTA's part [lo, hi) of a row in shared memory: element e lies at at(e), as far from a 16-byte
// boundary as in global memory; places from hi to the end of its chunk hold -inf.
template <typename E>
struct Stage {
  char* mem;         // 16-byte aligned, 16 spare bytes at both ends
  int lo, hi;
  uint32_t lead;     // the part's offset from a 16-byte boundary
  __device__ __forceinline__ char* at(int e) const { return mem + lead + (e - lo) * static_cast<int>(sizeof(E)); }
  __device__ __forceinline__ bool has(int e) const { return e >= lo && e < hi; }
  __device__ __forceinline__ uint16_t* word(int e) const { return reinterpret_cast<uint16_t*>(at(e)); }
  // One warp: whole 16-byte words by a bulk copy, the ends element by element.  The row that lay here
  // was read and in places written by plain accesses; the fence orders the copy behind them.
  __device__ __forceinline__ void fetch(const E* z, uint64_t* bar) const {
    const int lane = threadIdx.x & 31;
    fence_proxy_async_smem();
    __syncwarp();
    const int bytes = (hi - lo) * static_cast<int>(sizeof(E));
    const int head = min(bytes, static_cast<int>((16u - lead) & 15u)), body = (bytes - head) & ~15;
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, body);
      if (body > 0) bulk_load(mem + lead + head, reinterpret_cast<const char*>(z + lo) + head, body, bar);
    }
    const int h = head / sizeof(E), tl = (bytes - head - body) / sizeof(E);
    const int e = lane < h ? lo + lane : hi - tl + lane - h;
    if (lane < h + tl) *reinterpret_cast<E*>(at(e)) = z[e];
    if (lane < ((lo - hi) & 7)) store_one(reinterpret_cast<E*>(at(hi + lane)), -INFINITY);
  }
};

// The chunk at byte address p of shared memory, `shift` bytes past a 16-byte boundary.
template <typename E>
__device__ __forceinline__ Chunk<E> shared_chunk(const char* p, uint32_t shift) {
  if (shift != 0) return join_words<E>([&](int i) { return reinterpret_cast<const uint4*>(p - shift)[i]; }, shift);
  Chunk<E> c;
#pragma unroll
  for (int i = 0; i < Chunk<E>::kQ; ++i) c.set(i, reinterpret_cast<const uint4*>(p)[i]);
  return c;
}

// What a warp tells the other CTAs of a row about a slice.
struct alignas(16) Message {
  float m, s;
  int twice, unused;
};
// Sixteen bytes into the shared memory of CTA `rank` of the cluster, counted by its barrier: no fence, and
// so no waiting for the stores of the row before.
__device__ __forceinline__ void send(const void* slot, uint64_t* bar, int rank, const Message& m) {
  uint32_t a, b;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(slot)), "r"(rank));
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a),
               "r"(__float_as_uint(m.m)), "r"(__float_as_uint(m.s)), "r"(m.twice), "r"(0), "r"(b)
               : "memory");
}

struct BackwardSmem {
  Message part[2][kMaxSlices][kVocabWarps];   // by the parity of the row's number
  ListSmem list[2];
  RowResult result;
  int dead;
  uint64_t arrived[2];   // a slice of logits in a stage
  uint64_t joined[2];    // the messages of a row
  int abort;
};

struct BackwardPlan {
  int rows;          // consecutive rows a cluster
  int64_t T;
  int stages;        // 1 or 2 parts of rows in shared memory
  int stage_bytes;
};

constexpr int kBackwardThreads = kVocabThreads + 32;
enum : int { kBarArrived = 1, kBarResult = 2, kBarWritten = 3 };
__device__ __forceinline__ void bar_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kBackwardThreads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kBackwardThreads) : "memory");
}

// Loss and gradient.  A cluster takes `rows` consecutive rows, one after the other; a CTA of it has the
// same slices of each.  Eight warps go over the slices; a ninth serves them: it starts the
// copies, waits for them and for the other CTAs' sums (only one warp spins), finishes a row's
// scalars, and reads and reduces the next row's list meanwhile.  The CTAs of a row exchange
// their sums by asynchronous stores into each other's shared memory; the buffers alternate,
// because a CTA may be one row ahead of another, and no more: it needs that one's sums to go on.
template <typename E, bool kTail, bool kStage>
__global__ void __launch_bounds__(kBackwardThreads, 4) distill_topk_backward_kernel(const DistillArgs a,
                                                                                 const BackwardPlan plan) {
  constexpr int Q = Chunk<E>::kQ;
  extern __shared__ __align__(128) uint8_t dyn[];   // the stages, or the marks of two rows
  __shared__ BackwardSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool serves = warp == kVocabWarps;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / ctas) * plan.rows;
  const int n_rows = static_cast<int>(min(static_cast<int64_t>(plan.rows), plan.T - t0));
  const int slices = vocab_slices(a.V), mine = slices / ctas, s0 = rank * mine;
  const float c1 = a.scale * kLog2e;
  const int per = (((a.V + 7) >> 3) + slices - 1) / slices;
  int first, end, unused;
  slice_range(a.V, slices, s0, first, unused);
  slice_range(a.V, slices, s0 + mine - 1, unused, end);
  const int lo = min(a.V, 8 * first), hi = min(a.V, 8 * end);
  const int mark_words = kStage ? 0 : mine * Marks::slice_words(per);
  const auto marks_of = [&](int i) {
    return Marks{reinterpret_cast<unsigned*>(dyn) + (i & 1) * mark_words, first, per, end - first};
  };
  const auto z_of = [&](int i) { return static_cast<const E*>(a.logits) + (t0 + i) * a.ld; };
  const auto stage_of = [&](int i) {
    const E* z = z_of(i);
    return Stage<E>{reinterpret_cast<char*>(dyn) + (plan.stages == 2 ? i & 1 : 0) * plan.stage_bytes + 16, lo, hi,
                    static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z + lo)) & 15u};
  };
  const auto bar_of = [&](int i) { return &sm.arrived[plan.stages == 2 ? i & 1 : 0]; };

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.arrived[i], 1);
      mbar_init(&sm.joined[i], 1);
    }
    fence_mbar_init();
    sm.abort = 0;
  }
  if (!kStage)
    for (int i = tid; i < 2 * mark_words; i += kBackwardThreads) marks_of(0).words[i] = 0;
  cluster.sync();   // the barriers of every CTA are made; the marks are clear

  if (serves) {
    ListRegs<E, kTail> list;
    // row i's slices are there, its list is reduced: the others may begin
    // (a copy or a message that never comes leaves a status)
    const auto open_row = [&](int i) {
      if (kStage) {
        mbar_wait(bar_of(i), (plan.stages == 2 ? i >> 1 : i) & 1, a.status, &sm.abort);
        __syncwarp();   // the row's ends came by plain stores of single lanes; take_out's lanes write over them
        const bool twice = list.take_out(stage_of(i));
        if (lane == 0) sm.list[i & 1].twice = twice;
        __syncwarp();
      }
      bar_arrive(kBarArrived);
    };
    if (kStage)
      for (int i = 0; i < plan.stages && i < n_rows; ++i) stage_of(i).fetch(z_of(i), bar_of(i));
    // a single stage is free for the next row only at this one's end; till then L2 takes it (no further row:
    // two ahead cost 815 us where one gives 709)
    if (lane == 0 && kStage && plan.stages == 1 && n_rows > 1) prefetch_row(z_of(1), lo, hi);
    list.read(a, t0);
    list.gather(a, z_of(0));
    list.template reduce<!kStage>(a.scale, marks_of(0), sm.list[0]);
    open_row(0);
    for (int i = 0; i < n_rows; ++i) {
      const int64_t t = t0 + i;
      const ListSmem& l = sm.list[i & 1];
      const bool more = i + 1 < n_rows, dead = l.bad || !l.live;
      if (lane == 0) mbar_arrive_expect_tx(&sm.joined[i & 1], slices * kVocabWarps * sizeof(Message));
      if (kStage && plan.stages == 2 && i > 0 && more) stage_of(i + 1).fetch(z_of(i + 1), bar_of(i + 1));
      if (more) {   // the next row's list, while the others sum
        list.read(a, t + 1);
        if (!kStage && i > 0) list.clear(sm.list[(i + 1) & 1], marks_of(i + 1));
        list.gather(a, z_of(i + 1));
        list.template reduce<!kStage>(a.scale, marks_of(i + 1), sm.list[(i + 1) & 1]);
      }
      mbar_wait_cluster(&sm.joined[i & 1], (i >> 1) & 1, a.status, &sm.abort);   // messages of other CTAs are read next
      const Message* flat = &sm.part[i & 1][0][0];
      const int n = slices * kVocabWarps;
      Stats x = empty_stats(), y = empty_stats();
      bool twice = false;
      if (lane < n) {
        const Message g = flat[lane];
        x = {g.m, g.s, 0.f};
        twice |= g.twice != 0;
      }
      if (lane + 32 < n) {
        const Message g = flat[lane + 32];
        y = {g.m, g.s, 0.f};
        twice |= g.twice != 0;
      }
      const bool bad = l.bad || __any_sync(0xffffffffu, twice);
      const Stats st = Running<E, false>::join_two(x, y, c1);
      const RowResult r = finish_row<kTail>(st, l, c1);
      if (lane == 0) {
        sm.result = r;
        sm.dead = dead || bad;
      }
      __syncwarp();
      bar_arrive(kBarResult);
      if (rank == 0 && lane == 0) {
        const RowLoss o = row_loss<kTail>(st, r, l, a.scale);
        if (bad) set_status(a.status, kStatusBadInput);
        a.loss[t] = bad ? NAN : dead ? 0.f : o.loss;
        if (a.lse != nullptr) a.lse[t] = dead || bad ? 0.f : o.lse;
      }
      if (more && plan.stages == 2) open_row(i + 1);
      bar_sync(kBarWritten);   // the row's stage is free
      if (more && plan.stages == 1) {
        if (kStage) {
          stage_of(i + 1).fetch(z_of(i + 1), bar_of(i + 1));
          if (lane == 0 && i + 2 < n_rows) prefetch_row(z_of(i + 2), lo, hi);
        }
        open_row(i + 1);
      }
    }
    return;
  }

  for (int i = 0; i < n_rows; ++i) {
    const int64_t t = t0 + i;
    const E* z = z_of(i);
    const ListSmem& l = sm.list[i & 1];
    const Marks marks = marks_of(i);
    const Stage<E> stage = stage_of(i);
    const float w = a.scale * (a.dloss != nullptr ? a.dloss[t] : 1.f);
    bar_sync(kBarArrived);
    if (kStage) mbar_wait(bar_of(i), (plan.stages == 2 ? i >> 1 : i) & 1, a.status, &sm.abort);   // (it has come)
    const bool idle = l.bad || !l.live;
    for (int s = s0; s < s0 + mine; ++s) {
      Running<E, false> run;
      if (!idle) {
        int f, e;
        slice_range(a.V, slices, s, f, e);
        if (kStage) {
          const char* p = stage.at(8 * f);
          const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
          for (int c = tid; c < e - f; c += 4 * kVocabThreads) {
            Chunk<E> raw[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              raw[k] = shared_chunk<E>(p + 16 * Q * min(c + k * kVocabThreads, e - f - 1), shift);
            run.add(raw, e - f - c, c1);
          }
        } else {
          for_batches(Row<E>(static_cast<const E*>(a.logits), a.ld, t, a.V), f, e,
                      [&](int c, Chunk<E>(&raw)[4], int left) {
                        if (kTail) leave_out(raw, marks.batch(s - s0, c - f));
                        run.add(raw, left, c1);
                      });
        }
      }
      const Stats st = run.warp(c1);
      if (lane < ctas) send(&sm.part[i & 1][s][warp], &sm.joined[i & 1], lane, Message{st.m, st.s, l.twice, 0});
    }
    bar_sync(kBarResult);
    const RowResult r = sm.result;
    const bool dead = sm.dead;
    E* out = static_cast<E*>(a.dlogits) + t * a.ldd;
    const F2 cc = pack2(c1, c1), kk = pack2(w * r.coef, w * r.coef);
    const auto gradient = [&](int, const Chunk<E>& z8, float(&v)[8]) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 p = unpack2(mul2(z8.pair_minus(x, r.mb), cc));
        const float2 d = unpack2(mul2(pack2(ex2(p.x), ex2(p.y)), kk));
        v[2 * x] = d.x;
        v[2 * x + 1] = d.y;
      }
    };
    const auto zero = [](int, const Chunk<E>&, float(&v)[8]) {
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = 0.f;
    };
    if (dead) {
      map_chunks<E, 1>(out, lo, hi, [](int) { return Chunk<E>::none(); }, [&](int e) { return z[e]; }, zero);
    } else if (kStage) {
      // the shift of every chunk: out + e is on a boundary
      const uint32_t shift = (stage.lead - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(out + lo))) & 15u;
      map_chunks<E, 2>(out, lo, hi, [&](int e) { return shared_chunk<E>(stage.at(e), shift); },
                       [&](int e) { return *reinterpret_cast<const E*>(stage.at(e)); }, gradient);
    } else {
      map_row<E, 2>(z, a.V, out, lo, hi, gradient);
    }
    // the listed tokens' values go over the others (the list is read before its place is free)
    int id = -1;
    float listed = 0.f;
    if (!dead && tid < a.K) {
      id = l.id[tid];
      listed = listed_gradient(l, tid, r, c1, w);
    }
    bar_sync(kBarWritten);
    if (id >= lo && id < hi) store_one(out + id, listed);
  }
}

constexpr int kMaxSmem = 200 * 1024;     // dynamic: the stages and the marks

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), std::atomic<bool>* smem_set, int smem_max, int64_t ctas, int cluster,
                   int threads, int smem, cudaStream_t s, const Args&... args) {
  const cudaError_t e = set_smem_attr_once(smem_set, reinterpret_cast<const void*>(kernel), smem_max);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename E, bool kTail>
cudaError_t forward(const DistillArgs& a, int64_t T, cudaStream_t s) {
  static std::atomic<bool> set[64];
  const int slices = vocab_slices(a.V), chunks = (a.V + 7) / 8;
  int ctas = 1;
  while (ctas < slices && T * ctas < 4 * num_sms()) ctas *= 2;   // as the log probabilities
  const int words = slices / ctas * Marks::slice_words((chunks + slices - 1) / slices);
  return launch(distill_topk_kernel<E, kTail>, set, kMaxSmem, T * ctas, ctas, kVocabThreads, 4 * words, s, a);
}

constexpr int kStageAim = 66 * 1024;     // of a CTA's stages; three CTAs fit on an SM

template <typename E, bool kTail>
cudaError_t backward(const DistillArgs& a, int64_t T, cudaStream_t s) {
  static std::atomic<bool> set[2][64];
  const int slices = vocab_slices(a.V), per = ((a.V + 7) / 8 + slices - 1) / slices;
  const auto stage_bytes = [&](int n) {   // 16 spare bytes at both ends, 16 for the part's offset
    return static_cast<int64_t>(n) * per * 8 * sizeof(E) + 48;
  };
  // Slices a CTA: as many as a stage of the size aimed at takes, so that the work of a row that does not
  // grow with V is shared by few CTAs, while there are rows enough to fill the GPU.
  // (2048 x 131072 BF16: two slices a CTA 199 us, one 238 us, four 328 us.)
  int mine = 1;
  while (2 * mine <= slices && stage_bytes(2 * mine) <= kStageAim && T * (slices / (2 * mine)) >= 3 * num_sms())
    mine *= 2;
  const int ctas = slices / mine;
  BackwardPlan plan{};
  plan.T = T;
  plan.rows = 1;
  plan.stages = 1;
  if (stage_bytes(mine) <= kMaxSmem) {
    plan.stage_bytes = static_cast<int>(stage_bytes(mine));
    // Rows a cluster: one, for the hardware to balance, two where there are clusters enough all the same
    // (8192 x 131072 BF16: one 767 us, two 709 us, four 724 us; 1000 x 50021 float16: 54, 57, 57 us).  Where
    // whole rows are so short that two stages fit, several, so that the next row arrives meanwhile
    // (4096 x 8000 BF16: eight 39 us, one 47 us; longer rows do not gain).
    if (T * ctas >= 16 * num_sms()) plan.rows = 2;
    if (ctas == 1 && 2 * plan.stage_bytes <= kStageAim) {
      const int64_t rows = T / (4 * num_sms());
      plan.rows = static_cast<int>(rows < 1 ? 1 : rows > 8 ? 8 : rows);
      plan.stages = plan.rows > 1 ? 2 : 1;
    }
    return launch(distill_topk_backward_kernel<E, kTail, true>, set[0], kMaxSmem,
                  (T + plan.rows - 1) / plan.rows * ctas, ctas, kBackwardThreads, plan.stages * plan.stage_bytes, s, a,
                  plan);
  }
  const int marks = 2 * 4 * mine * Marks::slice_words(per);   // of two rows
  return launch(distill_topk_backward_kernel<E, kTail, false>, set[1], kMaxSmem, T * ctas, ctas, kBackwardThreads, marks,
                s, a, plan);
}

template <typename E>
cudaError_t dispatch(const DistillArgs& a, int64_t T, bool tail, cudaStream_t s) {
  if (a.dlogits != nullptr) return tail ? backward<E, true>(a, T, s) : backward<E, false>(a, T, s);
  return tail ? forward<E, true>(a, T, s) : forward<E, false>(a, T, s);
}

}  // namespace

cudaError_t launch_distill_topk(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld, const int32_t* ids,
                                const float* values, int K, bool tail, float scale, const float* dloss, float* loss,
                                float* lse, void* dlogits, int64_t ldd, cudaStream_t s) {
  DistillArgs a{logits, ld, static_cast<int>(V), ids, values, K, scale, dloss, loss, lse, dlogits, ldd,
                device_status_ptr()};
  if (dtype == kActBF16) return dispatch<__nv_bfloat16>(a, T, tail, s);
  if (dtype == kActF16) return dispatch<__half>(a, T, tail, s);
  return dispatch<float>(a, T, tail, s);
}

}  // namespace nvfp4
