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

#include "paged.cuh"

namespace clsample {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kLoad = 128;    // vectors that a warp loads at once
constexpr int kBatch = 256;  // vectors of a warp between two marks: at most 32 batches, a thread a vector
constexpr int kMaxVocab = 262144;

// floor(2^40 p) for p in [0, 1], as hi 2^23 + lo, hi = floor(2^17 p) and lo = floor(2^23 times
// the rest).  Adding 2^23 and truncating leaves an integer below 2^23 in a float's low bits;
// the rest is exact.  Four float32 operations, on two numbers at once: a conversion to 64 bits
// would run in the float64 unit, whose rate here bounds a call at four times the memory's time.
constexpr int kIntBits = 0x4b000000;  // of 2^23
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
struct Mass2 {
  int hi[2], lo[2];  // with kIntBits added to each
  __device__ __forceinline__ Mass2(float p0, float p1) {
    const uint64_t p = two(p0, p1), k17 = two(131072.f, 131072.f), k23 = two(8388608.f, 8388608.f);
    const uint64_t minus = two(-1.f, -1.f);
    uint64_t y, rest, z;
    asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(p), "l"(k17), "l"(k23));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(rest) : "l"(y), "l"(minus), "l"(k23));  // -hi
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(rest) : "l"(p), "l"(k17), "l"(rest));
    asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(z) : "l"(rest), "l"(k23), "l"(k23));
    asm("mov.b64 {%0, %1}, %2;" : "=r"(hi[0]), "=r"(hi[1]) : "l"(y));
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo[0]), "=r"(lo[1]) : "l"(z));
  }
};
__device__ __forceinline__ int64_t mass_of(int hi, int lo) { return ((int64_t)hi << 23) + lo; }

__device__ __forceinline__ bool bad_prob(float p) { return !(p >= 0.f && p <= 1.f); }

// Whether any of the probabilities seen was outside [0, 1] or NaN.
struct Range {
  float lo = 0.f, hi = 0.f;
  __device__ __forceinline__ void see(float p, float q) {
    asm("min.f32 %0, %0, %1, %2;" : "+f"(lo) : "f"(p), "f"(q));
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(hi) : "f"(p), "f"(q));  // keeps a NaN
  }
  __device__ __forceinline__ bool bad() const { return !(lo >= 0.f && hi <= 1.f); }
};

__device__ __forceinline__ float load_prob(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_prob(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }

__device__ __forceinline__ void widen16(const uint32_t (&w)[4], float (&x)[4], const float*) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void widen16(const uint32_t (&w)[4], float (&x)[8], const __nv_bfloat16*) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Pair<__nv_bfloat16>::widen(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <class P>
__device__ __forceinline__ int misaligned(const P* row) {  // elements past a 16-byte boundary
  return (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(P));
}

// What is drawn from: the target row, less the draft's row (q) or less everything at one
// token (hole), or neither.  The row is taken in 16-byte vectors that are aligned in p: vector
// v has the tokens v N - a .. v N - a + N - 1, a = misaligned(p), those of them that exist.  q
// may be aligned otherwise: its vector is then put together from the two that hold it.
template <class P>
struct Weights {
  static constexpr int N = 16 / sizeof(P);
  const P* p;
  const P* q;
  int hole, V, a, turn;  // turn: elements by which q's vectors lie later than p's
  __device__ __forceinline__ void set(const P* p_row, const P* q_row, int hole_at, int vocab) {
    p = p_row;
    q = q_row;
    hole = hole_at;
    V = vocab;
    a = misaligned(p);
    turn = q ? (misaligned(q) - a) & (N - 1) : 0;
  }
  __device__ __forceinline__ int vectors() const { return (V + a + N - 1) / N; }
  // vectors whose loads stay within the rows, in p and in q
  __device__ __forceinline__ int whole_from() const { return (a + turn + N - 1) / N; }
  __device__ __forceinline__ int whole_to() const { return max(0, (V + a - (turn ? N - turn : 0)) / N); }

  // 16 bytes of a row from token t0 on, of which the aligned vector before starts `shift` earlier
  __device__ __forceinline__ uint4 bits(const P* row, int t0, int shift) const {
    const uint4* at = reinterpret_cast<const uint4*>(row + t0 - shift);
    const uint4 v = __ldg(at);
    if (shift == 0) return v;
    const uint4 u = __ldg(at + 1);
    uint32_t z[9] = {v.x, v.y, v.z, v.w, u.x, u.y, u.z, u.w, 0};
    const int bytes = shift * (int)sizeof(P);
    if (bytes & 8)
#pragma unroll
      for (int i = 0; i < 7; ++i) z[i] = z[i + 2];
    if (bytes & 4)
#pragma unroll
      for (int i = 0; i < 7; ++i) z[i] = z[i + 1];
    const int b = (bytes & 2) * 8;
    return make_uint4(__funnelshift_r(z[0], z[1], b), __funnelshift_r(z[1], z[2], b), __funnelshift_r(z[2], z[3], b),
                      __funnelshift_r(z[3], z[4], b));
  }
  __device__ __forceinline__ void unpack(uint4 v, float (&x)[N]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    widen16(w, x, p);
  }
  // a vector's tokens one by one, those that there are
  __device__ __forceinline__ void edge(const P* row, int t0, float (&x)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = t0 + i >= 0 && t0 + i < V ? load_prob(row + t0 + i) : 0.f;
  }
  __device__ __forceinline__ void values(int v, float (&x)[N], float (&y)[N]) const {
    const int t0 = v * N - a;
    if (v >= whole_from() && v < whole_to()) {
      unpack(bits(p, t0, 0), x);
      if (q) unpack(bits(q, t0, turn), y);
    } else {
      edge(p, t0, x);
      if (q) edge(q, t0, y);
    }
  }
  // The weights' sum.  Where p > q, P >= Q, and elsewhere P <= Q.
  __device__ __forceinline__ int64_t sum_of(int v, const float (&x)[N], const float (&y)[N], Range* range) const {
    int hi = 0, lo = 0;  // of at most eight weights
    if (q) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        range->see(x[i], y[i]);
        range->see(x[i + 1], y[i + 1]);
        const Mass2 mp(x[i], x[i + 1]), mq(y[i], y[i + 1]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (x[i + e] > y[i + e]) {
            hi += mp.hi[e] - mq.hi[e];
            lo += mp.lo[e] - mq.lo[e];
          }
      }
    } else {
      const int t0 = v * N - a;
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        range->see(x[i], x[i + 1]);
        const Mass2 mp(x[i], x[i + 1]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (t0 + i + e != hole) {
            hi += mp.hi[e] - kIntBits;
            lo += mp.lo[e] - kIntBits;
          }
      }
    }
    return mass_of(hi, lo);
  }
  __device__ __forceinline__ void vector(int v, int64_t (&w)[N]) const {
    float x[N], y[N];
    values(v, x, y);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const Mass2 mp(x[i], x[i + 1]), mq(q ? y[i] : 0.f, q ? y[i + 1] : 0.f);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w[i + e] = (q && x[i + e] <= y[i + e]) || v * N - a + i + e == hole
                       ? 0
                       : mass_of(mp.hi[e] - mq.hi[e], mp.lo[e] - mq.lo[e]);
    }
  }
  // Sum over a warp's vectors first .. end - 1, kLoad at a time with four loads of each row in
  // flight; the lane's sum of each batch is left in marks[batch * kThreads].
  __device__ __forceinline__ int64_t sum_range(int first, int end, Range* range, int64_t* marks) const {
    const int lane = threadIdx.x & 31, from = whole_from(), to = min(end, whole_to());
    int64_t total = 0, sum = 0;
    for (int v0 = first; v0 < end; v0 += kLoad) {  // uniform over the warp
      if (v0 >= from && v0 + kLoad <= to) {
        uint4 x4[4], y4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x4[k] = bits(p, (v0 + 32 * k + lane) * N - a, 0);
        if (q) {
#pragma unroll
          for (int k = 0; k < 4; ++k) y4[k] = bits(q, (v0 + 32 * k + lane) * N - a, turn);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x[N], y[N];
          unpack(x4[k], x);
          unpack(y4[k], y);
          sum += sum_of(v0 + 32 * k + lane, x, y, range);
        }
      } else {
#pragma unroll 1
        for (int v = v0 + lane; v < min(end, v0 + kLoad); v += 32) {
          float x[N], y[N];
          values(v, x, y);
          sum += sum_of(v, x, y, range);
        }
      }
      if (v0 + kLoad >= end || (v0 + kLoad - first) % kBatch == 0) {
        *marks = sum;
        marks += kThreads;
        total += sum;
        sum = 0;
      }
    }
    return total;
  }
};

__device__ __forceinline__ int64_t warp_total(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

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

// Shared memory for the marks: a row may take one vector more than its tokens fill.
template <class P, int C>
int marks_bytes(int V) {
  constexpr int N = 16 / sizeof(P);
  const int vectors = (V + 2 * N - 2) / N, share = (vectors + C - 1) / C, part = (share + kWarps - 1) / kWarps;
  return (part + kBatch - 1) / kBatch * kThreads * (int)sizeof(int64_t);
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
