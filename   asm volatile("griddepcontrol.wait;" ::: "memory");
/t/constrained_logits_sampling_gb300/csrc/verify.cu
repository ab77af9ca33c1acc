// clsample_verify: drafted tokens against the target's probabilities (rule in
// include/clsample.h).
//
// One cluster of CTAs per request.  Every CTA takes the accept decisions for itself (a few
// gathered words), then sums the integer weights of its contiguous slice of the row to draw
// from, each warp a contiguous part; the slices' sums meet in distributed shared memory, and
// the CTA whose slice holds the threshold reads the part that holds it once more, a vector a
// thread, for the token.  Weights are integers, so the token does not depend on the split.
// Bound by memory: one row of p, and one of q after a refusal, are read once from HBM.
// 256 requests of 3 drafted tokens, 151936 float32 probabilities a row (245 MB read): 50 us, 4.9
// TB/s; about 3 us of it is the chain of loads before a row is known.
#include <cooperative_groups.h>

#include "draw_weights.cuh"

namespace clsample {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = kDrawThreads;

struct Shared {
  int64_t slice_sum[kMaxCluster];  // written by the cluster's CTAs
  int slice_bad[kMaxCluster];
  int64_t warp_sum[kWarps], scan[kWarps];
  int first;  // first refused drafted token, or n
  int bad;    // of the request; not written after it has been read
  int odd;    // a probability out of range in the CTA's slices: a warp may set it while another reads `bad`
};

template <class P, int C>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) verify_kernel(const __grid_constant__ clsample_verify_args_t a) {
  using W = Weights<P>;
  constexpr int N = W::N;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ Shared sh;
  extern __shared__ int64_t marks[];  // each thread's sums of its warp's batches
  // a CTA's shared memory may be written from afar only once it has started
  cluster.barrier_arrive();

  const int lo = __ldg(a.cu_draft + b), hi = __ldg(a.cu_draft + b + 1);
  const float u_last = __ldg(a.u_sample + b);
  const int n = hi - lo;
  bool bad = lo < 0 || hi < lo || hi > a.N || n > a.max_draft || !(u_last >= 0.f && u_last < 1.f);
  if (tid == 0) {
    sh.first = n;
    sh.bad = sh.odd = 0;
  }
  __syncthreads();
  const P* target = reinterpret_cast<const P*>(a.target);
  const P* draft = reinterpret_cast<const P*>(a.draft);
  if (!bad) {
    for (int i = tid; i < n; i += kThreads) {
      const int x = __ldg(a.draft_tokens + lo + i);
      const float u = __ldg(a.u_accept + lo + i);
      if (x < 0 || x >= a.V || !(u >= 0.f && u < 1.f)) {
        bad = true;
        continue;
      }
      const float p = load_prob(target + ((int64_t)lo + b + i) * a.target_stride + x);
      const float q = draft ? load_prob(draft + (int64_t)(lo + i) * a.draft_stride + x) : 1.f;
      bad |= bad_prob(p) || bad_prob(q);
      // both factors have 24 bits, so the 64-bit product is exact
      if (!((double)u * (double)q < (double)p)) atomicMin(&sh.first, i);
    }
  }
  if (bad) atomicOr(&sh.bad, 1);
  __syncthreads();
  bad = sh.bad;
  const int acc = sh.first;
  const bool refused = acc < n;
  cluster.barrier_wait();

  W w{};
  int64_t total = 0, before = 0;
  int begin = 0, end = 0, part = 0;  // the slice's vectors, and how many of them a warp has
  if (!bad) {  // uniform over the cluster: every CTA took the same decisions
    w.set(target + ((int64_t)lo + b + acc) * a.target_stride,
          refused && draft ? draft + (int64_t)(lo + acc) * a.draft_stride : nullptr,
          refused && !draft ? __ldg(a.draft_tokens + lo + acc) : -1, a.V);
    for (int pass = 0; pass < 2; ++pass) {
      const int share = (w.vectors() + C - 1) / C;
      begin = min(w.vectors(), rank * share);
      end = min(w.vectors(), begin + share);
      part = (share + kWarps - 1) / kWarps;
      const int w0 = min(end, begin + warp * part), w1 = min(end, w0 + part);
      Range range;
      const int64_t sum = warp_total(w.sum_range(w0, w1, &range, marks + tid));
      const bool odd = __any_sync(~0u, range.bad());
      if (lane == 0) {
        sh.warp_sum[warp] = sum;
        if (odd) atomicOr(&sh.odd, 1);
      }
      __syncthreads();
      if (tid < C) {
        int64_t mine = 0;
        for (int i = 0; i < kWarps; ++i) mine += sh.warp_sum[i];
        Shared* other = cluster.map_shared_rank(&sh, tid);
        other->slice_sum[rank] = mine;
        other->slice_bad[rank] = sh.odd;
      }
      cluster.sync();
      total = before = 0;
      for (int i = 0; i < C; ++i) {
        if (i < rank) before += sh.slice_sum[i];
        total += sh.slice_sum[i];
        bad |= sh.slice_bad[i] != 0;
      }
      if (total > 0 || bad || (!w.q && w.hole < 0)) break;
      // nothing of p is above q: draw from p itself
      w.set(w.p, nullptr, -1, a.V);
      cluster.sync();  // the sums have been read by all before they are written again
    }
    bad |= total == 0;
  }

  int32_t* out = a.tokens + (int64_t)b * a.token_stride;
  if (rank == 0) {
    for (int i = tid; i <= a.max_draft; i += kThreads)
      if (bad || i != acc) out[i] = !bad && i < acc ? __ldg(a.draft_tokens + lo + i) : -1;
    if (tid == 0) {
      if (a.accepted) a.accepted[b] = bad ? 0 : acc;
      if (a.row_status) a.row_status[b] = bad ? CLSAMPLE_ROW_INVALID : CLSAMPLE_ROW_OK;
    }
  }
  if (bad) return;
  // floor(u31 total / 2^31) with total below 2^58
  const int64_t u31 = __float2ll_rz(u_last * 2147483648.f);
  const int64_t k = u31 * (total >> 31) + ((u31 * (total & 0x7fffffff)) >> 31);
  int64_t left = k - before;
  if (left < 0 || left >= sh.slice_sum[rank]) return;  // another slice's
  int at = 0;  // the warp whose part holds the threshold
  while (left >= sh.warp_sum[at]) left -= sh.warp_sum[at++];
  // the batch of that warp: lane i adds up batch i
  int p0 = begin + at * part;
  const int p1 = min(end, p0 + part);
  const int batches = (p1 - p0 + kBatch - 1) / kBatch;  // at most 32
  int64_t run = 0;
  if (lane < batches)
#pragma unroll 8
    for (int i = 0; i < 32; ++i) run += marks[lane * kThreads + at * 32 + (i + lane) % 32];
  const int64_t batch_sum = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(~0u, run, o);
    if (lane >= o) run += up;
  }
  const int batch = __ffs(__ballot_sync(~0u, run > left)) - 1;
  left -= __shfl_sync(~0u, run - batch_sum, batch);
  p0 += batch * kBatch;
  // the token, a vector a thread
  static_assert(kBatch == kThreads, "one round");
  const int v = p0 + tid;
  int64_t x[N], mine = 0;
  if (v < p1) {
    w.vector(v, x);
#pragma unroll
    for (int i = 0; i < N; ++i) mine += x[i];
  }
  run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(~0u, run, o);
    if (lane >= o) run += up;
  }
  if (lane == 31) sh.scan[warp] = run;
  __syncthreads();
  for (int i = 0; i < warp; ++i) run += sh.scan[i];
  if (run > left && run - mine <= left) {
    int64_t c = run - mine;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (c <= left && left < c + x[i]) out[acc] = v * N - w.a + i;
      c += x[i];
    }
  }
}

template <class P, int C>
cudaError_t launch_verify(const clsample_verify_args_t& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.B * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)marks_bytes<P, C>(a.V);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaFuncSetAttribute(verify_kernel<P, C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             marks_bytes<P, C>(kMaxVocab));
  return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, verify_kernel<P, C>, a) : e;
}

// The largest cluster with which all requests are resident at once: one wave, each request
// over as many SMs as that leaves it.  256 requests over 151936 tokens: 50 us on 2 CTAs each, 53
// on 4, 61 on 8; one over 32000: 7.4 to 8.0 us on 8, 8.4 on 4, 10.3 on 2.
template <class P>
cudaError_t launch_verify(const clsample_verify_args_t& a, int sms, cudaStream_t st) {
  const int64_t slots = (int64_t)sms * kCtasPerSm;
  if (a.B * (int64_t)8 <= slots) return launch_verify<P, 8>(a, st);
  if (a.B * (int64_t)4 <= slots) return launch_verify<P, 4>(a, st);
  return launch_verify<P, 2>(a, st);
}

}  // namespace
}  // namespace clsample

extern "C" int clsample_verify(const clsample_verify_args_t* a, clsample_stream_t stream) {
  using namespace clsample;
  if (!a) return CLSAMPLE_ERR_NULL;
  if (a->B < 0 || a->B > (1 << 24) - 1 || a->N < 0) return CLSAMPLE_ERR_BATCH;
  if (a->V <= 0 || a->V > kMaxVocab) return CLSAMPLE_ERR_VOCAB;
  if (a->dtype != CLSAMPLE_LOGITS_F32 && a->dtype != CLSAMPLE_LOGITS_BF16) return CLSAMPLE_ERR_DTYPE;
  if (a->max_draft < 0) return CLSAMPLE_ERR_SHAPE;
  if (a->target_stride < a->V || (a->draft && a->draft_stride < a->V) || a->token_stride <= a->max_draft)
    return CLSAMPLE_ERR_STRIDE;
  if (a->B == 0) return CLSAMPLE_SUCCESS;
  if (!a->target || !a->cu_draft || !a->u_sample || !a->tokens || (a->N > 0 && (!a->draft_tokens || !a->u_accept)))
    return CLSAMPLE_ERR_NULL;
  int sms = 0;
  const int rc = check_device(nullptr, &sms);
  if (rc != CLSAMPLE_SUCCESS) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      a->dtype == CLSAMPLE_LOGITS_F32 ? launch_verify<float>(*a, sms, st) : launch_verify<__nv_bfloat16>(*a, sms, st);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? CLSAMPLE_SUCCESS : CLSAMPLE_ERR_CUDA;
}
