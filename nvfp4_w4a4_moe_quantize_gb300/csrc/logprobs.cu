// Log probabilities of given tokens, entropy and the top alternatives of rows of logits, and
// their backward.
//
//   c = scale z,  lse = ln sum exp(c),  logprob = c_y - lse,  H = lse - sum p c,  p = exp(c - lse)
//   dz = scale (g (1[j = y] - p) - h p (ln p + H))
//
// Forward: one pass over the row with a running maximum (vocab.cuh).
// The top k come out of the same pass.  Every thread leaves the maximum of each of its batches of 32
// elements (a cell).  The k-th best of the threads' own maxima is a lower bound of the k-th best
// of the row, so only cells that reach it can hold one of the top k; their few chunks are
// read again (from L2) and every element that reaches the bound becomes a candidate, ranked by
// (value, lowest id).  A sort or a heap over the row is not needed, and no atomic decides an
// order: a candidate's key is its value and id.
//
// Bound: HBM for the pass (8192 x 131072 BF16, a tenth of the rows ignored: 288 us, 6.7 TB/s of the
// rows read; backward 616 us, 7.0 TB/s read and written); what a list adds is latency at the end of
// a row, hidden behind the other three CTAs of the SM in part (2048 x 131072: no list 93 us, 20
// entries 120 us, 128 entries 135 us; of a row's 66000 cycles the bound takes 2400, the cells 1800, reading
// them again 7200, the sort 2900).  One row is bound by latency: 131072 BF16 logits over the 8 CTAs
// of a cluster with 20 entries 10 us.
#include "launch.h"
#include "status.cuh"
#include "vocab.cuh"

namespace nvfp4 {
namespace {

namespace cg = cooperative_groups;

constexpr int kCandidates = 1024;   // room for candidates; few more than k are usual
constexpr int kKeep = 512;          // when they do not fit: kept from round to round,
constexpr int kRound = 16;          // and batches read a round, at most 32 candidates each
constexpr int kMaxCells = 16;       // a thread
static_assert(kKeep + 32 * kRound <= kCandidates && kMaxList <= kKeep, "a round has to fit");
static_assert(sizeof(Stats) == 12, "a cluster's sums are 24 KB at most");
static_assert(kMaxSlices * kMaxList <= kCandidates, "the lists of a cluster have to fit");

// Order of the values as unsigned words; -0 counts as 0.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
// Larger value first, then the lower position.
__device__ __forceinline__ uint64_t order_key(float v, uint32_t pos) {
  return (static_cast<uint64_t>(order_bits(v)) << 32) | (0xffffffffu - pos);
}

struct LogprobSmem {
  Stats part[kVocabWarps];
  int count, cells;
  uint64_t bound;
};
struct TopSmem {
  float best[kMaxCells][kVocabThreads];       // a cell's best value, -inf: nothing there
  float thread_best[kVocabThreads];
  uint16_t cell[kMaxCells * kVocabThreads];   // cells that reach the bound
  alignas(16) uint64_t key[kCandidates + 8];
  uint64_t sorted[kMaxList];
  uint64_t lists[kMaxSlices][kMaxList];       // the cluster's lists (first CTA)
  int sizes[kMaxSlices];
};

// A CTA's slices [s0, s0 + mine) as cells: cell number s * per_slice + b of a thread is its batches
// [b * batches, (b + 1) * batches) of slice s0 + s.
struct Cells {
  int V, slices, s0, batches, per_slice;
  __device__ Cells(int V_, int slices_, int s0_, int mine) : V(V_), slices(slices_), s0(s0_) {
    int first, last;
    slice_range(V, slices, 0, first, last);   // no slice is longer than the first
    const int n = (last + 4 * kVocabThreads - 1) / (4 * kVocabThreads);
    batches = (mine * n + kMaxCells - 1) / kMaxCells;
    per_slice = (n + batches - 1) / batches;  // mine per_slice <= kMaxCells: 16 / mine is whole
  }
  // first chunk of batch j of a thread's cell; last: the end of its slice
  __device__ __forceinline__ int chunk(int cell, int thread, int j, int& last) const {
    const int s = cell / per_slice;
    int first;
    slice_range(V, slices, s0 + s, first, last);
    return first + thread + ((cell - s * per_slice) * batches + j) * 4 * kVocabThreads;
  }
};

// One key a thread, in descending order over the CTA: a bitonic network, exchanges between warps through buf.
__device__ __forceinline__ uint64_t sort_keys(uint64_t x, uint64_t* buf) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int k = 2; k <= kVocabThreads; k *= 2)
#pragma unroll
    for (int j = k / 2; j > 0; j /= 2) {
      uint64_t y;
      if (j < 32) {
        y = __shfl_xor_sync(0xffffffffu, x, j);
      } else {
        buf[tid] = x;
        __syncthreads();
        y = buf[tid ^ j];
        __syncthreads();
      }
      const bool larger = ((tid & j) == 0) == ((tid & k) == 0);
      x = (x > y) == larger ? x : y;
    }
  return x;
}

// The best min(n, k) of key[0 .. n) in order into out; returns how many.  Keys differ, so a
// key's rank is the number of larger ones; that costs n steps a key, a sort 36, so the sort takes
// over where a warp is not enough for the keys.  key has room for 8 more than n.
__device__ __forceinline__ int rank_keys(uint64_t* key, int n, int k, uint64_t* out) {
  if (n > 48 && n <= kVocabThreads) {
    const uint64_t mine = threadIdx.x < n ? key[threadIdx.x] : 0;
    __syncthreads();
    const uint64_t x = sort_keys(mine, key);
    if (threadIdx.x < min(n, k)) out[threadIdx.x] = x;
    __syncthreads();
    return min(n, k);
  }
  if (threadIdx.x < 8) key[n + threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kVocabThreads) {
    const uint64_t mine = key[i];
    int rank = 0;
    for (int j = 0; j < n; j += 8) {
      ulonglong2 two[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) two[x] = reinterpret_cast<const ulonglong2*>(key + j)[x];
#pragma unroll
      for (int x = 0; x < 4; ++x) rank += (two[x].x > mine) + (two[x].y > mine);
    }
    if (rank < k) out[rank] = mine;
  }
  __syncthreads();
  return min(n, k);
}

// A lower bound of the row's k-th best key, from the threads' best values (`mine`); the whole CTA.
// 0 when fewer than k threads hold anything, or hardly more (n <= enough): every allowed element then is a
// candidate, where they do not fit in rounds.
//   The values are searched bit by bit for a bound that at least k threads reach, until hardly
//   more do: every bit costs a vote of the CTA, and a few candidates too many cost less.
__device__ __forceinline__ uint64_t list_bound(float mine, TopSmem& t, const Cells& cells, int n_cells, int k,
                                               uint64_t* plateau) {
  const uint32_t val = mine > -INFINITY ? order_bits(mine) : 0u;
  t.thread_best[threadIdx.x] = mine;
  int n = __syncthreads_count(val != 0);
  if (n < k) return 0;
  uint32_t v = 0;
  const int enough = k + (k >> 3) + 4;
  for (int bit = 31; bit >= 0 && n > enough; --bit) {
    const uint32_t next = v | (1u << bit);
    const int m = __syncthreads_count(val >= next);
    if (m >= k) {
      v = next;
      n = m;
    }
  }
  if (n <= 2 * enough) return static_cast<uint64_t>(v) << 32;
  // Many share one value (a plateau; v is exact, every bit was searched): the lowest places are searched for
  // in the same way, by one warp.  A thread has that value no later than in the last chunk of its
  // first cell that reaches it.
  if (threadIdx.x < 32) {
    const float value = order_value(v);
    uint32_t chunk[kVocabWarps];
    int over = 0;
#pragma unroll
    for (int w = 0; w < kVocabWarps; ++w) {
      const int i = w * 32 + threadIdx.x;
      over += t.thread_best[i] > value;
      int q = 0, last;
      while (q + 1 < n_cells && t.best[q][i] != value) ++q;
      chunk[w] = t.thread_best[i] == value ? cells.chunk(q, i, cells.batches - 1, last) + 3 * kVocabThreads : ~0u;
    }
    over = __reduce_add_sync(0xffffffffu, over);
    uint32_t c = 0xfffffu;
    for (int b = 19; b >= 0; --b) {
      const uint32_t next = c & ~(1u << b);
      int m = 0;
#pragma unroll
      for (int w = 0; w < kVocabWarps; ++w) m += chunk[w] <= next;
      if (over + __reduce_add_sync(0xffffffffu, m) >= k) c = next;
    }
    if (threadIdx.x == 0) *plateau = (static_cast<uint64_t>(v) << 32) | (0xffffffffu - (8 * c + 7));
  }
  __syncthreads();
  return *plateau;
}

struct LogprobArgs {
  const void* logits;
  int64_t ld;
  int V;
  const int32_t* targets;
  int32_t ignore;
  float scale;
  int k;
  float *logprob, *lse, *entropy, *top_logprob;
  int32_t* top_ids;
  int* status;
};

// One row a cluster of 1, 2, 4 or 8 CTAs; a CTA runs its part of the row's slices in turn.
template <typename E, bool kEntropy, bool kTop>
__global__ void __launch_bounds__(kVocabThreads, kTop || sizeof(E) == 4 ? 4 : 6)
    token_logprobs_kernel(const LogprobArgs a) {
  extern __shared__ __align__(16) uint8_t dyn[];   // TopSmem; a cluster's sums, by slice and thread
  __shared__ LogprobSmem sm;
  TopSmem& top = *reinterpret_cast<TopSmem*>(dyn);
  Stats* slice_sums = reinterpret_cast<Stats*>(dyn + (kTop ? sizeof(TopSmem) : 0));
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int64_t t = blockIdx.x / ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (ctas > 1) cluster.barrier_arrive();   // met below, before another CTA's shared memory is written
  const int32_t y = a.targets != nullptr ? a.targets[t] : 0;
  if (a.targets != nullptr && y == a.ignore) {   // the same in every CTA of the cluster
    if (rank == 0) {
      if (tid == 0) {
        a.logprob[t] = 0.f;
        a.lse[t] = 0.f;
        if (kEntropy) a.entropy[t] = 0.f;
      }
      if (kTop)
        for (int i = tid; i < a.k; i += kVocabThreads) {
          a.top_logprob[t * a.k + i] = -INFINITY;
          a.top_ids[t * a.k + i] = -1;
        }
    }
    if (ctas > 1) cluster.barrier_wait();
    return;
  }
  const Row<E> row(static_cast<const E*>(a.logits), a.ld, t, a.V);
  const int slices = vocab_slices(a.V);
  const float c1 = a.scale * kLog2e;
  const int mine = slices / ctas, s0 = rank * mine, s1 = s0 + mine;
  const float zy = rank == 0 && tid == 0 && a.targets != nullptr && y >= 0 && y < a.V ? to_f32(row.p[y]) : 0.f;
  // A thread's sums of the slices are added in the slices' order, here or in the cluster's first CTA.
  Stats row_sums = empty_stats();
  Stats* lead_sums = ctas == 1 ? nullptr : cluster.map_shared_rank(slice_sums, 0);
  if (kTop && tid == 0) sm.count = sm.cells = 0;
  const Cells cells(a.V, slices, s0, mine);
  const int n_cells = mine * cells.per_slice;
  float thread_best = -INFINITY;
  for (int s = s0; s < s1; ++s) {
    int first, last;
    slice_range(a.V, slices, s, first, last);
    if (tid == 0 && s + 1 < s1) {   // the next slice on its way into L2: more bytes than the registers can await
      int f, l;
      slice_range(a.V, slices, s + 1, f, l);
      prefetch_row(row.p, min(a.V, 8 * f), min(a.V, 8 * l));
    }
    Running<E, kEntropy> run;
    if (kTop)   // the cells that this thread does not reach
      for (int q = 0; q < cells.per_slice; ++q) top.best[(s - s0) * cells.per_slice + q][tid] = -INFINITY;
    float best = -INFINITY;
    int q = (s - s0) * cells.per_slice, left_in_cell = cells.batches;
    for_batches(row, first, last, [&](int c, const Chunk<E>(&raw)[4], int left) {
      const float cm = run.add(raw, left, c1);
      if (kTop) {
        best = fmaxf(best, cm);
        top.best[q][tid] = best;
        if (--left_in_cell == 0) {
          thread_best = fmaxf(thread_best, best);
          best = -INFINITY;
          left_in_cell = cells.batches;
          ++q;
        }
      }
    });
    if (kTop) thread_best = fmaxf(thread_best, best);
    if (ctas == 1) {
      row_sums = Running<E, kEntropy>::join(row_sums, run.thread(), c1);
    } else {
      if (s == s0) cluster.barrier_wait();
      lead_sums[s * kVocabThreads + tid] = run.thread();
    }
  }
  if (ctas == 1) {   // (read after the list's barriers)
    row_sums = Running<E, kEntropy>::warp_join(row_sums, c1);
    if (lane == 0) sm.part[warp] = row_sums;
    if (!kTop) __syncthreads();
  }
  int found = 0;
  if (kTop) {
    const uint64_t bound = list_bound(thread_best, top, cells, n_cells, a.k, &sm.bound);
    const float floor = bound == 0 ? -INFINITY : order_value(static_cast<uint32_t>(bound >> 32));
    const bool plateau = static_cast<uint32_t>(bound) != 0;   // the key's lower half matters there alone
    // (one count a warp: many lanes at one counter would wait for each other)
    const auto reserve = [&](int* counter, int n, int& total) {   // places [returned, returned + n) of the counter
      int before = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, before, o);
        before += lane >= o ? x : 0;
      }
      total = __shfl_sync(0xffffffffu, before, 31);
      int base = 0;
      if (lane == 0 && total > 0) base = atomicAdd(counter, total);
      return __shfl_sync(0xffffffffu, base, 0) + before - n;
    };
    {
      unsigned hit = 0;
      if (thread_best >= floor && thread_best > -INFINITY)
#pragma unroll 4
        for (int q = 0; q < n_cells; ++q)
          if (top.best[q][tid] >= floor && top.best[q][tid] > -INFINITY) hit |= 1u << q;
      int total, at = reserve(&sm.cells, __popc(hit), total);
      for (; hit != 0; hit &= hit - 1)
        top.cell[at++] = static_cast<uint16_t>((__ffs(hit) - 1) * kVocabThreads + tid);
    }
    __syncthreads();
    // the cells' batches, a thread each
    const int items = sm.cells * cells.batches;
    const auto read = [&](int item, Chunk<E>(&raw)[4], int& c) {
      const int i = cells.batches == 1 ? item : item / cells.batches;
      const int cell = top.cell[i];
      int last;
      c = cells.chunk(cell / kVocabThreads, cell % kVocabThreads, item - i * cells.batches, last);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        raw[k] = c + k * kVocabThreads < last ? row.get(c + k * kVocabThreads) : Chunk<E>::none();
    };
    // the elements that reach the bound; every lane of a warp calls it
    const auto collect = [&](int item) {
      Chunk<E> raw[4];
      int c = 0;
      unsigned hit = 0;   // a bit an element
      if (item < items) {
        read(item, raw, c);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (raw[k].max() >= floor) {
            float v[8];
            unpack8(raw[k], v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (v[i] >= floor && v[i] > -INFINITY) hit |= 1u << (8 * k + i);
            if (plateau)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (order_key(v[i], 8 * (c + k * kVocabThreads) + i) < bound) hit &= ~(1u << (8 * k + i));
          }
      }
      int total, at = reserve(&sm.count, __popc(hit), total);
      if (total == 0) return;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        while (hit >> (8 * k) & 255u) {   // mostly one
          const int i = __ffs(hit >> (8 * k) & 255u) - 1;
          hit &= ~(1u << (8 * k + i));
          float v[8];
          unpack8(raw[k], v);
          float x = v[0];
#pragma unroll
          for (int j = 1; j < 8; ++j) x = j == i ? v[j] : x;
          if (at < kCandidates) top.key[at] = order_key(x, 8 * (c + k * kVocabThreads) + i);
          ++at;
        }
    };
    for (int base = 0; base < items; base += kVocabThreads) collect(base + tid);
    __syncthreads();
    if (sm.count > kCandidates) {   // too many (most of the large values lie in few cells): again, in rounds
      __syncthreads();
      if (tid == 0) sm.count = 0;
      for (int base = 0; base < items; base += kRound) {
        __syncthreads();
        if (warp == 0) collect(lane < kRound ? base + lane : items);
        __syncthreads();
        const int n = sm.count;
        if (n > kKeep) {            // keep the best k, so that the next round has room
          rank_keys(top.key, n, a.k, top.sorted);
          if (tid < a.k) top.key[tid] = top.sorted[tid];
          if (tid == 0) sm.count = a.k;
        }
      }
      __syncthreads();
    }
    found = rank_keys(top.key, sm.count, a.k, top.sorted);
    if (ctas > 1) {   // push the list into the first CTA
      TopSmem* lead = cluster.map_shared_rank(&top, 0);
      if (tid < found) lead->lists[rank][tid] = top.sorted[tid];
      if (tid == 0) lead->sizes[rank] = found;
    }
  }
  if (ctas > 1) {
    cluster.sync();
    if (rank != 0) return;
    for (int s = 0; s < slices; ++s)
      row_sums = Running<E, kEntropy>::join(row_sums, slice_sums[s * kVocabThreads + tid], c1);
    row_sums = Running<E, kEntropy>::warp_join(row_sums, c1);
    if (lane == 0) sm.part[warp] = row_sums;
    __syncthreads();
  }
  const Stats st =   // every warp, the same bits
      Running<E, kEntropy>::warp_join(lane < kVocabWarps ? sm.part[lane] : empty_stats(), c1);
  const float ln_s = logf(st.s);
  const bool none = st.s == 0.f;   // every token excluded
  if (tid == 0) {
    if (a.targets != nullptr) {
      float lp = -INFINITY;
      if (y < 0 || y >= a.V) {
        set_status(a.status, kStatusBadInput);
        lp = NAN;
      } else if (!none) {
        lp = fmaf(zy - st.m, a.scale, -ln_s);
      }
      a.logprob[t] = lp;
    }
    a.lse[t] = none ? -INFINITY : fmaf(st.m, a.scale, ln_s);
    if (kEntropy) {
      const float h = ln_s - kLn2 * (st.u / st.s);
      a.entropy[t] = none || h < 0.f ? 0.f : h;   // round-off below 0
    }
  }
  if (kTop) {
    if (ctas > 1) {
      // Merge the sorted lists.  If every list has k / ctas keys, k of them reach the smallest of
      // those lists' (k / ctas)-th keys, so few others remain to be ranked.
      const int share = (a.k + ctas - 1) / ctas;
      uint64_t least = ~uint64_t(0);
      for (int l = 0; l < ctas; ++l) {
        const uint64_t key = top.sizes[l] < share ? 0 : top.lists[l][share - 1];
        least = key < least ? key : least;
      }
      if (tid == 0) sm.count = 0;
      __syncthreads();
      for (int i = tid; i < ctas * kMaxList; i += kVocabThreads) {
        const int l = i / kMaxList, p = i % kMaxList;
        if (p < top.sizes[l] && top.lists[l][p] >= least) top.key[atomicAdd(&sm.count, 1)] = top.lists[l][p];
      }
      __syncthreads();
      found = rank_keys(top.key, sm.count, a.k, top.sorted);
    }
    for (int i = tid; i < a.k; i += kVocabThreads) {
      float lp = -INFINITY;
      int32_t id = -1;
      if (i < found) {
        lp = fmaf(order_value(static_cast<uint32_t>(top.sorted[i] >> 32)) - st.m, a.scale, -ln_s);
        id = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(top.sorted[i]));
      }
      a.top_logprob[t * a.k + i] = lp;
      a.top_ids[t * a.k + i] = id;
    }
  }
}

template <typename E, bool kEntropy, bool kTop>
cudaError_t launch_forward(const LogprobArgs& a, int64_t T, cudaStream_t s) {
  static std::atomic<bool> smem_set[64];
  const int slices = vocab_slices(a.V);
  // few rows: a row's slices in a cluster, over as many CTAs as it takes to fill the GPU
  int ctas = 1;
  while (ctas < slices && T * ctas < 4 * num_sms()) ctas *= 2;
  const int smem = (kTop ? static_cast<int>(sizeof(TopSmem)) : 0) +
                   (ctas > 1 ? static_cast<int>(sizeof(Stats)) * slices * kVocabThreads : 0);
  auto kernel = token_logprobs_kernel<E, kEntropy, kTop>;
  if (smem > 0) {
    const cudaError_t e = set_smem_attr_once(smem_set, reinterpret_cast<const void*>(kernel), 96 * 1024);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(T * ctas));
  cfg.blockDim = dim3(kVocabThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename E>
cudaError_t forward_dtype(const LogprobArgs& a, int64_t T, cudaStream_t s) {
  if (a.k > 0) return a.entropy ? launch_forward<E, true, true>(a, T, s) : launch_forward<E, false, true>(a, T, s);
  return a.entropy ? launch_forward<E, true, false>(a, T, s) : launch_forward<E, false, false>(a, T, s);
}

struct LogprobBackwardArgs {
  const void* logits;
  int64_t ld;
  int V;
  const int32_t* targets;
  int32_t ignore;
  float scale;
  const float *lse, *entropy, *dlogprob, *dentropy;
  void* dlogits;
  int64_t ldd;
  int tiles;
};

constexpr int kBackwardTile = 16384;   // elements of a row a CTA
constexpr float kLowestLse = -16777216.f;   // -2^24: below, float32 is 2 and more apart, and p = exp(c - lse) lost

// One exponential an element; the tiles are independent, so the loads of 4 chunks a thread and the CTAs of
// an SM cover the latency (8192 x 131072 BF16: 614 us, with the entropy 616 us, 6.97 TB/s, the rate of a copy).
template <typename E, bool kEntropy>
__global__ void __launch_bounds__(kVocabThreads) token_logprobs_backward_kernel(const LogprobBackwardArgs a) {
  const int64_t t = blockIdx.x / a.tiles;
  const int lo = static_cast<int>(blockIdx.x % a.tiles) * kBackwardTile, hi = min(a.V, lo + kBackwardTile);
  const E* z = static_cast<const E*>(a.logits) + t * a.ld;
  E* out = static_cast<E*>(a.dlogits) + t * a.ldd;
  const int32_t y = a.targets != nullptr ? a.targets[t] : -1;
  const float lse = a.lse[t];
  // a target that the forward refused adds nothing
  const float g = a.dlogprob != nullptr && y >= 0 && y < a.V ? a.dlogprob[t] : 0.f;
  const float h = kEntropy ? a.dentropy[t] : 0.f;
  // nothing to learn from the row: ignored, or nothing above a mask's values, lowest or -1e9 added to every
  // token (a lse of that size has lost ln s, and p with it)
  const bool skip = (a.targets != nullptr && y == a.ignore) || lse < kLowestLse;
  // with t = log2 p:  dz = p (A + B t), + scale g at the target.  ln p = scale z - lse is rounded once and
  // brought to base 2 after that: scale log2(e) and lse log2(e), rounded first, would each add a rounding of
  // lse's size to lse's own
  const float A = -a.scale * (g + (kEntropy ? h * a.entropy[t] : 0.f)), B = -a.scale * h * kLn2;
  const F2 cc = pack2(a.scale, a.scale), ll = pack2(-lse, -lse), to2 = pack2(kLog2e, kLog2e);
  const F2 aa = pack2(A, A), bb = pack2(B, B);
  const float zy = a.scale * g;
  map_row<E, 4>(z, a.V, out, lo, hi, [&](int e0, const Chunk<E>& z8, float(&v)[8]) {
    const unsigned at = y - e0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 lt = unpack2(mul2(fma2(z8.pair(i), cc, ll), to2));
      const F2 p = pack2(ex2(lt.x), ex2(lt.y));
      // 2^-1000 is 0: the clamp changes no product, and keeps 0 away from B * inf
      const F2 f = kEntropy ? fma2(bb, pack2(fmaxf(lt.x, -1000.f), fmaxf(lt.y, -1000.f)), aa) : aa;
      const float2 d = unpack2(mul2(p, f));
      v[2 * i] = d.x;
      v[2 * i + 1] = d.y;
    }
    if (at < 8) {   // the target, unless it is excluded
      float zv[8];
      unpack8(z8, zv);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i == at && zv[i] > -INFINITY) v[i] += zy;
    }
    if (skip)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
  });
}

template <typename E>
cudaError_t backward_dtype(const LogprobBackwardArgs& a, int64_t T, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(T * a.tiles));
  if (a.dentropy != nullptr) token_logprobs_backward_kernel<E, true><<<grid, kVocabThreads, 0, s>>>(a);
  else token_logprobs_backward_kernel<E, false><<<grid, kVocabThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_logprobs(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                                  const int32_t* targets, int32_t ignore, float scale, int k, float* logprob,
                                  float* lse, float* entropy, float* top_logprob, int32_t* top_ids, cudaStream_t s) {
  LogprobArgs a{logits, ld, static_cast<int>(V), targets, ignore, scale, k, logprob, lse, entropy, top_logprob,
                top_ids, device_status_ptr()};
  if (dtype == kActBF16) return forward_dtype<__nv_bfloat16>(a, T, s);
  if (dtype == kActF16) return forward_dtype<__half>(a, T, s);
  return forward_dtype<float>(a, T, s);
}

cudaError_t launch_token_logprobs_backward(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                                           const int32_t* targets, int32_t ignore, float scale, const float* lse,
                                           const float* entropy, const float* dlogprob, const float* dentropy,
                                           void* dlogits, int64_t ldd, cudaStream_t s) {
  LogprobBackwardArgs a{logits, ld, static_cast<int>(V), targets, ignore, scale, lse, entropy, dlogprob, dentropy,
                        dlogits, ldd, static_cast<int>((V + kBackwardTile - 1) / kBackwardTile)};
  if (dtype == kActBF16) return backward_dtype<__nv_bfloat16>(a, T, s);
  if (dtype == kActF16) return backward_dtype<__half>(a, T, s);
  return backward_dtype<float>(a, T, s);
}

}  // namespace nvfp4
