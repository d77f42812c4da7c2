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
// The gradient is 2^((z - m) scale log2 e) times one number of the row, and on S a value that is written
// over it afterwards.  The row is read twice, the second time from L2: the CTAs of a row are
// one cluster, so few rows are in flight and they stay there.
#include "launch.h"
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

struct DistillSmem {
  Stats part[kMaxSlices][kVocabWarps];
  int id[kMaxList];
  float red[4][kVocabWarps];
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
// Over the block, the same bits in every thread.
__device__ __forceinline__ float block_max(float x, float* red) {
  x = warp_max(x);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int w = 1; w < kVocabWarps; ++w) x = fmaxf(x, red[w]);
  __syncthreads();
  return x;
}
__device__ __forceinline__ float block_sum(float x, float* red) {
  x = warp_sum(x);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = red[0];
#pragma unroll
  for (int w = 1; w < kVocabWarps; ++w) x += red[w];
  __syncthreads();
  return x;
}

template <typename E, bool kTail, bool kGrad>
__global__ void __launch_bounds__(kVocabThreads) distill_topk_kernel(const DistillArgs a) {
  extern __shared__ __align__(16) uint8_t listed[];   // kTail: a byte a chunk of this CTA's slices
  __shared__ DistillSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int64_t t = blockIdx.x / ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Row<E> row(static_cast<const E*>(a.logits), a.ld, t, a.V);
  const int slices = vocab_slices(a.V);
  const float c1 = a.scale * kLog2e;
  const int s0 = ctas == 1 ? 0 : rank, s1 = ctas == 1 ? slices : rank + 1;
  int first, end, unused;
  slice_range(a.V, slices, s0, first, unused);
  slice_range(a.V, slices, s1 - 1, unused, end);

  // the teacher's list: an entry a thread (every CTA of the row computes the same)
  int id = -1;
  float tv = -INFINITY;
  bool bad = false;
  if (tid < a.K) {
    id = a.ids[t * a.K + tid];
    tv = a.values[t * a.K + tid];
    bad = id < -1 || id >= a.V;
    if (bad || id == -1) {
      id = -1;
      tv = -INFINITY;
    }
  }
  if (tid < kMaxList) sm.id[tid] = id;
  if (kTail)
    for (int i = tid; 16 * i < end - first; i += kVocabThreads)
      reinterpret_cast<uint4*>(listed)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  if (id >= 0)
    for (int j = 0; j < tid; ++j) bad |= sm.id[j] == id;
  bad = __syncthreads_or(bad);                     // an id outside [0, V) or twice in the row
  const bool live = __syncthreads_or(tv > -INFINITY || (kTail && id >= 0) || tv != tv);
  const E* z = row.p;
  const int lo = 8 * first, hi = min(a.V, 8 * end);
  E* out = kGrad ? static_cast<E*>(a.dlogits) + t * a.ldd : nullptr;
  if (bad || !live) {   // nothing to learn from the row; a bad row's loss is NaN
    if (rank == 0 && tid == 0) {
      if (bad) set_status(a.status, kStatusBadInput);
      a.loss[t] = bad ? NAN : 0.f;
      if (a.lse != nullptr) a.lse[t] = 0.f;
    }
    if (kGrad)
      for (int e = lo + tid; e < hi; e += kVocabThreads) store_one(out + e, 0.f);
    return;
  }
  if (ctas > 1) cluster.sync();   // every CTA of the cluster has started: its shared memory may be written
  if (kTail && id >= lo && id < hi)
    atomicOr(reinterpret_cast<unsigned*>(listed) + ((id - lo) >> 5), 1u << ((id - lo) & 31));
  const float zi = id >= 0 ? to_f32(z[id]) : -INFINITY;
  __syncthreads();

  // one pass over the row (the tokens outside the list, with the tail)
  for (int s = s0; s < s1; ++s) {
    int f, l;
    slice_range(a.V, slices, s, f, l);
    Stats st = empty_stats();
    for_chunks(row, f, l, [&](int c, float(&v)[8]) {
      if (kTail) {
        const uint32_t b = listed[c - first];
        if (b != 0)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (b >> i & 1) v[i] = -INFINITY;
      }
      accumulate<false>(st, v, c1);
    });
    st = warp_merge<false>(st, c1);
    if (lane == 0)
      for (int r = 0; r < (kGrad ? ctas : 1); ++r) {   // the gradient needs the sums in every CTA
        Stats(*part)[kVocabWarps] = ctas == 1 ? sm.part : cluster.map_shared_rank(sm.part, r);
        part[s][warp] = st;
      }
  }
  if (ctas > 1) {
    cluster.sync();
    if (!kGrad && rank != 0) return;
  } else {
    __syncthreads();
  }
  Stats st = join_slices<false>(sm.part, slices, c1);

  // Probabilities outside the list are k1 2^((c - mb) log2 e): mb is a maximum and k1 holds the
  // sum, so that rows of a mask's lowest values keep their digits.
  float mb, coef, m, ln_s, q, lq, qr = 0.f, lr = 0.f;   // lse = scale m + ln_s;  lr = ln p_r
  const bool rest = st.s != 0.f;   // some token outside the list is allowed (NaN counts)
  if (kTail) {
    mb = st.m;
    float on_m = -FLT_MAX, on_s = 0.f;
    if (zi > -INFINITY || zi != zi) {
      on_m = zi;
      on_s = zi < INFINITY ? 1.f : NAN;
    }
    // the list's own sum, over the block
    const float ln_rest = rest ? logf(st.s) : -INFINITY;
    m = fmaxf(block_max(on_m, sm.red[0]), st.m);
    const float sum = block_sum(on_s == 0.f ? 0.f : ex2((on_m - m) * c1) * on_s, sm.red[1]);
    const float rest_s = st.s;
    rebase<false>(st, m, c1);
    ln_s = logf(st.s + sum);
    lr = rest ? fmaf(mb - m, a.scale, ln_rest - ln_s) : -INFINITY;
    q = id >= 0 ? expf(tv) : 0.f;
    lq = tv;
    qr = fmaxf(0.f, 1.f - block_sum(q, sm.red[2]));
    coef = rest ? (expf(lr) - qr) / rest_s : 0.f;
  } else {
    mb = m = st.m;
    ln_s = logf(st.s);
    const float mt = block_max(tv, sm.red[0]);
    const float e = id >= 0 ? expf(tv - mt) : 0.f;
    const float sum = block_sum(e, sm.red[2]);
    q = e / sum;
    lq = tv - mt - logf(sum);
    coef = rest ? 1.f / st.s : 0.f;
  }
  const float lp = zi == -INFINITY ? -INFINITY : fmaf(zi - m, a.scale, -ln_s);
  const float term = id >= 0 && q != 0.f ? q * (lq - lp) : 0.f;
  float loss = block_sum(term, sm.red[3]);
  if (kTail && rest && qr > 0.f) loss += qr * (logf(qr) - lr);
  if (rank == 0 && tid == 0) {
    a.loss[t] = loss;
    if (a.lse != nullptr) a.lse[t] = fmaf(m, a.scale, ln_s);
  }
  if (kGrad) {
    const float w = a.scale * (a.dloss != nullptr ? a.dloss[t] : 1.f);
    const float k1 = w * coef;
    map_range(z, out, lo, hi, tid, kVocabThreads, [&](int, float(&v)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = k1 * ex2((v[i] - mb) * c1);
    });
    __syncthreads();
    if (id >= lo && id < hi) store_one(out + id, zi == -INFINITY ? 0.f : w * (expf(lp) - q));
  }
}

template <typename E, bool kTail, bool kGrad>
cudaError_t launch(const DistillArgs& a, int64_t T, cudaStream_t s) {
  static std::atomic<bool> smem_set[64];
  const int slices = vocab_slices(a.V);
  const int ctas = kGrad || T < 4 * num_sms() ? slices : 1;
  const int chunks = (a.V + 7) / 8;
  const int bytes = kTail ? (ctas == 1 ? chunks : (chunks + slices - 1) / slices) : 0;
  const int smem = (bytes + 15) / 16 * 16;
  auto kernel = distill_topk_kernel<E, kTail, kGrad>;
  if (kTail) {
    const cudaError_t e =
        set_smem_attr_once(smem_set, reinterpret_cast<const void*>(kernel), static_cast<int>(kMaxVocab / 8));
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
cudaError_t dispatch(const DistillArgs& a, int64_t T, bool tail, cudaStream_t s) {
  if (a.dlogits != nullptr) return tail ? launch<E, true, true>(a, T, s) : launch<E, false, true>(a, T, s);
  return tail ? launch<E, true, false>(a, T, s) : launch<E, false, false>(a, T, s);
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
