// clsample_verify: drafted tokens against the target's probabilities (rule in
// include/clsample.h).
//
// One cluster of CTAs per request.  Every CTA takes the accept decisions for itself (a few
// gathered words), then sums the integer weights of its contiguous slice of the row to draw
// from; the slices' sums meet in distributed shared memory, and the CTA whose slice holds
// the threshold reads it once more, warp by warp, for the token.  Weights are integers, so
// the token does not depend on the split.  Bound by memory: one row of p, and one of q
// after a refusal, are read once from HBM.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace clsample {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxVocab = 262144;

// 2^40 p as an integer for p in [0, 1]; the scaling is exact, the conversion truncates.
__device__ __forceinline__ int64_t mass_of(float p) { return __float2ll_rz(p * 1099511627776.f); }

__device__ __forceinline__ bool bad_prob(float p) { return !(p >= 0.f && p <= 1.f); }

__device__ __forceinline__ float load_prob(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_prob(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }

// What is drawn from: the target row, less the draft's row (q) or less everything at one
// token (hole), or neither.
template <class P>
struct Weights {
  const P* p;
  const P* q;
  int hole;
  __device__ __forceinline__ int64_t at(int t, bool* bad) const {
    const float x = load_prob(p + t);
    *bad |= bad_prob(x);
    int64_t w = mass_of(x);
    if (q) {
      const float y = load_prob(q + t);
      *bad |= bad_prob(y);
      w = max(w - mass_of(y), (int64_t)0);
    }
    return t == hole ? 0 : w;
  }
};

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

struct Shared {
  int64_t slice_sum[kCluster];  // written by the cluster's CTAs
  int slice_bad[kCluster];
  int64_t warp_sum[kWarps];
  int first;  // first refused drafted token, or n
  int bad;
};

template <class P>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(clsample_verify_args_t a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int b = blockIdx.x / kCluster;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ Shared sh;
  // a CTA's shared memory may be written from afar only once it has started
  cluster.barrier_arrive();

  const int lo = __ldg(a.cu_draft + b), hi = __ldg(a.cu_draft + b + 1);
  const float u_last = __ldg(a.u_sample + b);
  const int n = hi - lo;
  bool bad = lo < 0 || hi < lo || hi > a.N || n > a.max_draft || !(u_last >= 0.f && u_last < 1.f);
  if (tid == 0) {
    sh.first = n;
    sh.bad = 0;
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
      const float p = load_prob(target + (int64_t)(lo + b + i) * a.target_stride + x);
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

  const int share = (a.V + kCluster - 1) / kCluster;
  const int s0 = min(a.V, rank * share), s1 = min(a.V, s0 + share);
  // each warp sums a contiguous part of the slice
  const int part = (s1 - s0 + kWarps - 1) / kWarps;
  const int w0 = min(s1, s0 + warp * part), w1 = min(s1, w0 + part);
  Weights<P> w{};
  int64_t total = 0, before = 0;
  if (!bad) {  // uniform over the cluster: every CTA took the same decisions
    w.p = target + (int64_t)(lo + b + acc) * a.target_stride;
    w.q = refused && draft ? draft + (int64_t)(lo + acc) * a.draft_stride : nullptr;
    w.hole = refused && !draft ? __ldg(a.draft_tokens + lo + acc) : -1;
    for (int pass = 0; pass < 2; ++pass) {
      int64_t sum = 0;
      bool odd = false;
      for (int t = w0 + lane; t < w1; t += 32) sum += w.at(t, &odd);
      sum = warp_sum(sum);
      odd = __any_sync(~0u, odd);
      if (lane == 0) {
        sh.warp_sum[warp] = sum;
        if (odd) atomicOr(&sh.bad, 1);
      }
      __syncthreads();
      if (tid < kCluster) {
        int64_t mine = 0;
        for (int i = 0; i < kWarps; ++i) mine += sh.warp_sum[i];
        Shared* other = cluster.map_shared_rank(&sh, tid);
        other->slice_sum[rank] = mine;
        other->slice_bad[rank] = sh.bad;
      }
      cluster.sync();
      total = before = 0;
      for (int i = 0; i < kCluster; ++i) {
        if (i < rank) before += sh.slice_sum[i];
        total += sh.slice_sum[i];
        bad |= sh.slice_bad[i] != 0;
      }
      if (total > 0 || bad || (!w.q && w.hole < 0)) break;
      // nothing of p is above q: draw from p itself
      w.q = nullptr;
      w.hole = -1;
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
  for (int i = 0; i < warp; ++i) left -= sh.warp_sum[i];
  if (left < 0 || left >= sh.warp_sum[warp]) return;  // another warp's
  for (int t0 = w0; t0 < w1; t0 += 32) {
    bool odd = false;
    const int64_t v = t0 + lane < w1 ? w.at(t0 + lane, &odd) : 0;
    int64_t run = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(~0u, run, o);
      if (lane >= o) run += up;
    }
    const unsigned above = __ballot_sync(~0u, run > left);
    if (above) {
      if (lane == __ffs(above) - 1) out[acc] = t0 + lane;
      return;
    }
    left -= __shfl_sync(~0u, run, 31);
  }
}

template <class P>
cudaError_t launch_verify(const clsample_verify_args_t& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.B * kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kCluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<P>, a);
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
  const int rc = check_device();
  if (rc != CLSAMPLE_SUCCESS) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      a->dtype == CLSAMPLE_LOGITS_F32 ? launch_verify<float>(*a, st) : launch_verify<__nv_bfloat16>(*a, st);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? CLSAMPLE_SUCCESS : CLSAMPLE_ERR_CUDA;
}
