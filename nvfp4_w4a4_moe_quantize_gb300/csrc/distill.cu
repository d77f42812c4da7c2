// Distillation from a teacher's top logits: a row's loss over the student's logits z, and its
// gradient in the same call.
//
//   c = scale z, lse = ln sum exp(c), p = exp(c - lse);  S = the teacher's list, values t
//   tail off: q = softmax(t over S);   tail on: q = exp(t), q_r = max(0, 1 - sum q)
//   L = sum_S q (ln q - (c - lse))  [+ q_r (ln q_r - ln p_r), p_r = the student's mass outside S]
//   dL/dc = p - q on S;  outside p, or with the tail p - q_r p / p_r = exp(c - lse_r) (p_r - q_r)
//
// With the tail, the sum over the tokens outside S is taken on its own, with its own running
// maximum (a bitmap of S in shared memory, one byte a chunk, leaves them out): 1 - sum_S p
// would cancel when the student's mass lies on S.  lse then is that of the two parts.
// The gradient is 2^((z - m) scale log2 e) times one number of the row, and on S a value that
// is written over it afterwards.
// One warp of each CTA reduces the list to a few sums while the row arrives; the row's
// maximum enters them afterwards, so nothing but scalars follows the exchange.
// With the gradient, a row's slices are a cluster, a CTA each, and a slice stays in shared memory
// between the sum and the gradient: the row is read once.  A slice too long for that is
// read again.
#include <type_traits>

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
// A = sum q ln q, B = sum q (z - mz), Q = sum q.
struct ListSmem {
  int id[kMaxList];
  float q[kMaxList], z[kMaxList];
  float mz, s, A, B, Q;
  int live, bad;
};
// What the row's sums give: the loss, and the gradient as coef 2^((z - mb) c1), lp(z) = ln p.
struct RowResult {
  float loss, lse, mb, coef;
  float m, ln_s;
};
struct DistillSmem {
  Stats part[kMaxSlices][kVocabWarps];
  int twice[kMaxSlices];   // a slice found an id of the list twice
  ListSmem list;
  RowResult result;
  uint64_t arrived;
  int abort, dead;
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

// One warp: reads row t's list, marks those of its ids that lie in [lo, hi) in `listed`, which
// every thread of the CTA has cleared before `sync`, and leaves the sums in sm.
template <typename E, bool kTail, typename Sync>
__device__ __forceinline__ void reduce_list(const DistillArgs& a, const E* z, int64_t t, int lo, int hi,
                                            unsigned* listed, ListSmem& sm, int& twice, Sync&& sync) {
  constexpr int N = kMaxList / 32;
  const int lane = threadIdx.x & 31;
  const float c1 = a.scale * kLog2e;
  int id[N];
  float v[N], zi[N];
  bool bad = false, live = false;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int i = lane + 32 * j;
    id[j] = i < a.K ? a.ids[t * a.K + i] : -1;
    v[j] = i < a.K ? a.values[t * a.K + i] : -INFINITY;
    if (id[j] < 0 || id[j] >= a.V) {
      bad |= id[j] != -1;
      id[j] = -1;
      v[j] = -INFINITY;
    }
    zi[j] = id[j] >= 0 ? to_f32(z[id[j]]) : -INFINITY;
    live |= kTail ? id[j] >= 0 : !(v[j] == -INFINITY);   // NaN lives
  }
  sync();
  bool again = false;
  float mv = -INFINITY, mz = -FLT_MAX;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (id[j] >= lo && id[j] < hi) {
      const unsigned bit = 1u << ((id[j] - lo) & 31);
      again |= (atomicOr(listed + ((id[j] - lo) >> 5), bit) & bit) != 0;
    }
    mv = fmaxf(mv, v[j]);
    mz = fmaxf(mz, zi[j]);
  }
  mz = warp_max(mz);
  if (!kTail) mv = warp_max(mv);
  float e[N], esum = 0.f, s = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    e[j] = id[j] >= 0 ? expf(kTail ? v[j] : v[j] - mv) : 0.f;
    esum += e[j];
    if (!(zi[j] == -INFINITY)) s += ex2((zi[j] - mz) * c1);
  }
  esum = warp_sum(esum);
  const float ln_e = kTail ? 0.f : logf(esum);
  float A = 0.f, B = 0.f, Q = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float q = kTail ? e[j] : e[j] / esum;
    if (q != 0.f) {   // 0 ln 0 = 0
      A += q * (kTail ? v[j] : v[j] - mv - ln_e);
      B += q * (zi[j] - mz);
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
    twice = any_twice;
  }
}

template <bool kTail>
__device__ __forceinline__ RowResult finish_row(Stats st, const ListSmem& l, float scale, float c1) {
  RowResult r;
  const bool rest = st.s != 0.f;   // some token outside the list is allowed (NaN counts)
  r.mb = st.m;
  float tail = 0.f;
  if (kTail) {
    const float rest_s = st.s, ln_rest = rest ? logf(st.s) : -INFINITY;
    r.m = fmaxf(l.mz, st.m);
    rebase<false>(st, r.m, c1);
    st.s += l.s == 0.f ? 0.f : ex2((l.mz - r.m) * c1) * l.s;
    r.ln_s = logf(st.s);
    const float lr = rest ? fmaf(r.mb - r.m, scale, ln_rest - r.ln_s) : -INFINITY;   // ln p_r
    const float qr = fmaxf(0.f, 1.f - l.Q);
    r.coef = rest ? (expf(lr) - qr) / rest_s : 0.f;
    if (rest && qr > 0.f) tail = qr * (logf(qr) - lr);
  } else {
    r.m = st.m;
    r.ln_s = logf(st.s);
    r.coef = rest ? 1.f / st.s : 0.f;
  }
  // sum q (ln q - ln p) with ln p = scale (z - m) - ln s; a student without any allowed token
  // has p = 0 everywhere
  if (l.Q == 0.f) r.loss = tail;
  else if (st.s == 0.f) r.loss = INFINITY;
  else r.loss = l.A - scale * (l.B + l.Q * (l.mz - r.m)) + r.ln_s * l.Q + tail;
  r.lse = fmaf(r.m, scale, r.ln_s);
  return r;
}

// The listed tokens of a batch, four bytes of the bitmap 256 apart, become -inf.
template <bool kTail, typename E>
__device__ __forceinline__ void leave_out(Chunk<E> (&raw)[4], const uint8_t* listed, int chunks_left) {
  if constexpr (kTail) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t bits = k * kVocabThreads < chunks_left ? listed[k * kVocabThreads] : 0;
      if (bits != 0)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (bits >> i & 1) raw[k].leave_out(i);
    }
  }
}

// The loss alone.
template <typename E, bool kTail>
__global__ void __launch_bounds__(kVocabThreads) distill_topk_kernel(const DistillArgs a) {
  extern __shared__ __align__(16) uint8_t listed[];   // a byte a chunk of this CTA's slices
  __shared__ DistillSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int64_t t = blockIdx.x / ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (ctas > 1) cluster.barrier_arrive();   // met below, before anything is written to another CTA
  const Row<E> row(static_cast<const E*>(a.logits), a.ld, t, a.V);
  const int slices = vocab_slices(a.V);
  const float c1 = a.scale * kLog2e;
  const int s0 = ctas == 1 ? 0 : rank, s1 = ctas == 1 ? slices : rank + 1;
  int first, end, unused;
  slice_range(a.V, slices, s0, first, unused);
  slice_range(a.V, slices, s1 - 1, unused, end);
  for (int i = tid; 16 * i < end - first; i += kVocabThreads)
    reinterpret_cast<uint4*>(listed)[i] = make_uint4(0, 0, 0, 0);
  if (warp == 0)
    reduce_list<E, kTail>(a, row.p, t, 8 * first, 8 * end, reinterpret_cast<unsigned*>(listed), sm.list,
                          sm.twice[rank], [] { __syncthreads(); });
  else
    __syncthreads();
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
        leave_out<kTail>(raw, listed + (c - first), left);
        run.add(raw, left, c1);
      });
      const Stats st = run.warp(c1);
      if (lane == 0) *(ctas == 1 ? &sm.part[s][warp] : cluster.map_shared_rank(&sm.part[s][warp], 0)) = st;
    }
  if (ctas > 1) {
    if (tid == 0 && rank != 0) *cluster.map_shared_rank(&sm.twice[rank], 0) = sm.twice[rank];
    cluster.sync();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }
  if (warp != 0) return;
  bool bad = l.bad;
  for (int r = 0; r < ctas; ++r) bad |= sm.twice[r] != 0;
  RowResult r{0.f, 0.f};
  if (!dead) r = finish_row<kTail>(Running<E, false>::join_slices(sm.part, slices, c1), l, a.scale, c1);
  if (lane == 0) {
    if (bad) set_status(a.status, kStatusBadInput);
    a.loss[t] = bad ? NAN : r.loss;
    if (a.lse != nullptr) a.lse[t] = bad ? 0.f : r.lse;
  }
}

// A CTA's slice of a row in shared memory: element e of [lo, hi) lies at at(e), as far from a
// 16-byte boundary as in global memory.
template <typename E>
struct Stage {
  const char* mem;   // 16-byte aligned, 16 spare bytes at both ends
  int lo, hi;
  uint32_t lead;     // the slice's offset from a 16-byte boundary
  __device__ __forceinline__ const char* at(int e) const { return mem + lead + (e - lo) * static_cast<int>(sizeof(E)); }
  // Starts the copy: whole 16-byte words by one bulk copy, the ends by the first threads.
  __device__ __forceinline__ void fetch(const E* z, uint64_t* bar) const {
    const int bytes = (hi - lo) * static_cast<int>(sizeof(E));
    const char* g = reinterpret_cast<const char*>(z + lo);
    char* s = const_cast<char*>(mem) + lead;
    const int head = min(bytes, static_cast<int>((16u - lead) & 15u)), body = (bytes - head) & ~15;
    if (threadIdx.x == 0) {
      mbar_arrive_expect_tx(bar, body);
      if (body > 0) bulk_load(s + head, g + head, body, bar);
    }
    const int h = head / sizeof(E), tl = (bytes - head - body) / sizeof(E);
    const int i = static_cast<int>(threadIdx.x) - 32;   // another warp than the one that issues the copy
    const int e = i < h ? lo + i : hi - tl + i - h;
    if (i >= 0 && i < h + tl) *reinterpret_cast<E*>(const_cast<char*>(at(e))) = z[e];
  }
  // Elements [e, e + 8).
  __device__ __forceinline__ Chunk<E> get(int e) const {
    constexpr int Q = Chunk<E>::kQ;
    const char* p = at(e);
    const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
    const uint4* w = reinterpret_cast<const uint4*>(p - shift);
    if (shift != 0) return join_words<E>([&](int i) { return w[i]; }, shift);
    Chunk<E> c;
#pragma unroll
    for (int i = 0; i < Q; ++i) c.set(i, w[i]);
    return c;
  }
};

template <typename E, bool kTail, bool kStage>
__global__ void __launch_bounds__(kVocabThreads) distill_topk_backward_kernel(const DistillArgs a, int stage_bytes) {
  extern __shared__ __align__(128) uint8_t dyn[];   // kStage: the slice; then a byte a chunk of it
  __shared__ DistillSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int64_t t = blockIdx.x / ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (ctas > 1) cluster.barrier_arrive();   // met below, before anything is written to another CTA
  const Row<E> row(static_cast<const E*>(a.logits), a.ld, t, a.V);
  const E* z = row.p;
  uint8_t* listed = dyn + stage_bytes;
  const float c1 = a.scale * kLog2e;
  int first, end;
  slice_range(a.V, ctas, rank, first, end);
  const int lo = min(a.V, 8 * first), hi = min(a.V, 8 * end);
  Stage<E> stage{reinterpret_cast<const char*>(dyn) + 16, lo, hi,
                 static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z + lo)) & 15u};
  if (kStage) {
    if (tid == 0) {
      mbar_init(&sm.arrived, 1);
      fence_mbar_init();
      sm.abort = 0;
    }
    stage.fetch(z, &sm.arrived);   // its first thread made the barrier
  }
  for (int i = tid; 16 * i < end - first; i += kVocabThreads)
    reinterpret_cast<uint4*>(listed)[i] = make_uint4(0, 0, 0, 0);
  if (warp == kVocabWarps - 1)
    reduce_list<E, kTail>(a, z, t, lo, hi, reinterpret_cast<unsigned*>(listed), sm.list, sm.twice[rank],
                          [] { __syncthreads(); });
  else
    __syncthreads();
  __syncthreads();
  const ListSmem& l = sm.list;
  if (kStage) mbar_wait(&sm.arrived, 0, a.status, &sm.abort);   // (a copy that never came leaves a status)
  bool dead = l.bad || !l.live;
  Stats st = empty_stats();
  if (!dead) {
    Running<E, false> run;
    if (kStage) {
      for (int c = first + tid; c < end; c += 4 * kVocabThreads) {
        Chunk<E> raw[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int ck = c + k * kVocabThreads;
          raw[k] = ck < end ? stage.get(8 * ck) : Chunk<E>::none();
          if (ck < end && 8 * ck + 8 > a.V)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (8 * ck + i >= a.V) raw[k].leave_out(i);
        }
        leave_out<kTail>(raw, listed + (c - first), end - c);
        run.add(raw, end - c, c1);
      }
    } else {
      for_batches(row, first, end, [&](int c, Chunk<E>(&raw)[4], int left) {
        leave_out<kTail>(raw, listed + (c - first), left);
        run.add(raw, left, c1);
      });
    }
    st = run.warp(c1);
  }
  if (ctas > 1) {
    cluster.barrier_wait();
    if (lane < ctas) {
      *cluster.map_shared_rank(&sm.part[rank][warp], lane) = st;
      if (warp == 0 && lane != rank) *cluster.map_shared_rank(&sm.twice[rank], lane) = sm.twice[rank];
    }
    cluster.sync();
  } else {
    if (lane == 0) sm.part[0][warp] = st;
    __syncthreads();
  }
  // one warp finishes the row's scalars for the CTA
  if (warp == 0) {
    bool bad = l.bad;
    for (int r = 0; r < ctas; ++r) bad |= sm.twice[r] != 0;
    RowResult r{0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (!dead) r = finish_row<kTail>(Running<E, false>::join_slices(sm.part, ctas, c1), l, a.scale, c1);
    if (bad) {
      r.loss = NAN;
      r.lse = 0.f;
    }
    if (lane == 0) {
      sm.result = r;
      sm.dead = dead || bad;
      if (rank == 0) {
        if (bad) set_status(a.status, kStatusBadInput);
        a.loss[t] = r.loss;
        if (a.lse != nullptr) a.lse[t] = r.lse;
      }
    }
  }
  __syncthreads();
  const RowResult r = sm.result;
  dead = sm.dead;
  const float w = a.scale * (a.dloss != nullptr ? a.dloss[t] : 1.f);
  E* out = static_cast<E*>(a.dlogits) + t * a.ldd;
  const F2 minus = pack2(-r.mb, -r.mb), cc = pack2(c1, c1), kk = pack2(w * r.coef, w * r.coef);
  const auto gradient = [&](int, float(&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack2(mul2(add2(pack2(v[2 * i], v[2 * i + 1]), minus), cc));
      const float2 d = unpack2(mul2(pack2(ex2(x.x), ex2(x.y)), kk));
      v[2 * i] = d.x;
      v[2 * i + 1] = d.y;
    }
    if (dead)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
  };
  if (kStage)
    map_chunks<E, 2>(out, lo, hi, [&](int e) { return stage.get(e); },
                     [&](int e) { return *reinterpret_cast<const E*>(stage.at(e)); }, gradient);
  else
    map_row<E, 2>(z, a.V, out, lo, hi, gradient);
  if (dead) return;
  __syncthreads();   // the listed tokens' values go over the others
  if (tid < kMaxList) {
    const int id = l.id[tid];
    const float zi = l.z[tid];
    if (id >= lo && id < hi)
      store_one(out + id, zi == -INFINITY ? 0.f : w * (expf(fmaf(zi - r.m, a.scale, -r.ln_s)) - l.q[tid]));
  }
}

template <typename K>
cudaError_t launch(K kernel, std::atomic<bool>* smem_set, int smem_max, int64_t ctas, int cluster, int smem,
                   cudaStream_t s, const DistillArgs& a, int stage) {
  const cudaError_t e = set_smem_attr_once(smem_set, reinterpret_cast<const void*>(kernel), smem_max);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kVocabThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if constexpr (std::is_invocable_v<K, DistillArgs, int>) return cudaLaunchKernelEx(&cfg, kernel, a, stage);
  else return cudaLaunchKernelEx(&cfg, kernel, a);
}

constexpr int kMaxSmem = 200 * 1024;   // a slice and its bitmap

template <typename E, bool kTail>
cudaError_t forward(const DistillArgs& a, int64_t T, cudaStream_t s) {
  static std::atomic<bool> set[64];
  const int slices = vocab_slices(a.V), chunks = (a.V + 7) / 8;
  const int ctas = T < 4 * num_sms() ? slices : 1;
  const int bytes = ctas == 1 ? chunks : (chunks + slices - 1) / slices;
  return launch(distill_topk_kernel<E, kTail>, set, static_cast<int>(kMaxVocab / 8), T * ctas, ctas,
                (bytes + 15) / 16 * 16, s, a, 0);
}

template <typename E, bool kTail>
cudaError_t backward(const DistillArgs& a, int64_t T, cudaStream_t s) {
  static std::atomic<bool> set[2][64];
  const int slices = vocab_slices(a.V), per = ((a.V + 7) / 8 + slices - 1) / slices;
  const int bits = (per + 15) / 16 * 16;
  const int64_t slice = static_cast<int64_t>(per) * 8 * sizeof(E) + 48;   // 16 spare bytes at both ends, 16 for its offset
  if (slice + bits <= kMaxSmem)
    return launch(distill_topk_backward_kernel<E, kTail, true>, set[0], kMaxSmem, T * slices, slices,
                  static_cast<int>(slice) + bits, s, a, static_cast<int>(slice));
  return launch(distill_topk_backward_kernel<E, kTail, false>, set[1], kMaxSmem, T * slices, slices, bits, s, a, 0);
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
