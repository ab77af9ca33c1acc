// clsample_verify_tree: a walk down a tree of drafted tokens (rule in include/clsample.h).
//
// One cluster of CTAs per request, as for clsample_verify.  Every CTA gathers what the walk needs of
// all drafted tokens at once (parents, ids, random numbers, p and q at the ids).  Its first warp then
// takes the decisions: a token is tried if its parent is the last accepted one, so the next to try is found
// by a ballot over the parents.  (All CTAs of a cluster take the same ones.  By all warps they cost 2 us a
// refusal, as exact comparisons run in the float64 unit.)  A refusal by a draft with probabilities needs
// the sum of what is left of the row: one pass of the cluster over p and q, whose sums meet in
// distributed shared memory; the last such pass is also the one that the token is drawn from.  As all
// refused children of a token came from one row q, what is left is max(P - Q c, 0) with one
// number c, and a pass costs the same after any number of refusals.  No pass is needed where the next
// child is accepted whatever the sum: s does not grow.
// A draft that is certain needs one pass, over the last token's row, with its refused ids as
// holes in a bitmap.  Bound by memory where requests are many: p and q once for each refusal on the
// path (256 requests of 6 refusals over 151936 tokens, 1.87 GB: 347 us, 5.4 TB/s); else by the chain of
// passes, each 4 us over 151936 tokens on 16 CTAs.
#include <cooperative_groups.h>

#include "draw_weights.cuh"

namespace clsample {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = kDrawThreads;
constexpr int kMaxNodes = 1023;
constexpr int kMaxCtas = 16;  // of a cluster

struct Shared {
  int64_t slice_sum[2][kMaxCtas];  // written by the cluster's CTAs, in passes by turns
  int slice_bad[2][kMaxCtas];
  int64_t warp_sum[kWarps], scan[kWarps];
  int bad;  // of the request; not written after it has been read
  int odd;  // a probability out of range in the CTA's slices
  int x[kMaxNodes + 1], row[kMaxNodes + 1], of_parent[kMaxNodes + 1];  // of_parent: the row of a token's children
  float u[kMaxNodes + 1], p[kMaxNodes + 1], q[kMaxNodes + 1];
  short parent[kMaxNodes + 1], path[kMaxNodes + 1];
  bool as_first[kMaxNodes + 1];  // accepted if it is its parent's first child
  // What the first warp has found: whose row to sum (or to draw from, if `end`), less which row how often.
  struct Step {
    int node, acc, refused, row;
    float taken;
    bool end;
  } step;
  // Where the walk stands between sums.  Here and not in registers, of which a thread has 64: what did not fit
  // went through local memory in every pass (256 requests of 6 refusals 375 us, 347 since).
  struct Walk {
    int at;        // the last token looked at
    float s, c;
    int64_t removed;
  } walk;
  int64_t total;  // of the last pass
};

__device__ __forceinline__ int64_t warp_total(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// floor(2^40 p), p in [0, 1]
__device__ __forceinline__ int64_t mass_at(float p) { return (int64_t)((double)p * 1099511627776.0); }
// m / 2^40 rounded to float32
__device__ __forceinline__ float share_of(int64_t m) { return __ll2float_rn(m) * 9.094947017729282379150390625e-13f; }

// A CTA's share of a row's vectors, and how many of them a warp has.
template <int C>
struct Share {
  int begin, end, part;
  __device__ __forceinline__ Share(int vectors, int rank) {
    const int share = (vectors + C - 1) / C;
    begin = min(vectors, rank * share);
    end = min(vectors, begin + share);
    part = (share + kWarps - 1) / kWarps;
  }
};

template <class P, int C>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    verify_tree_kernel(const __grid_constant__ clsample_verify_tree_args_t a) {
  using W = Weights<P, true>;
  constexpr int N = W::N;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ Shared sh;
  extern __shared__ int64_t marks[];  // each thread's sums of its warp's batches; then the holes
  // a CTA's shared memory may be written from afar only once it has started
  cluster.barrier_arrive();

  const int lo = __ldg(a.cu_draft + b), hi = __ldg(a.cu_draft + b + 1);
  const float u_last = __ldg(a.u_sample + b);
  bool bad = lo < 0 || hi < lo || hi > a.N || hi - lo > a.max_draft || !(u_last >= 0.f && u_last < 1.f);
  const int n = bad ? 0 : hi - lo;  // at most kMaxNodes
  if (tid == 0) {
    sh.bad = sh.odd = 0;
    sh.step = {-1, 0, 0, 0, 0.f, false};
    sh.walk = {-1, 1.f, 0.f, 0};
  }
  for (int i = tid; i <= n; i += kThreads) sh.of_parent[i] = -1;
  __syncthreads();
  const P* target = reinterpret_cast<const P*>(a.target);
  const P* draft = reinterpret_cast<const P*>(a.draft);
  const int64_t row0 = (int64_t)lo + b;  // the root's
  for (int i = tid; i < n; i += kThreads) {
    const int parent = __ldg(a.parents + lo + i), x = __ldg(a.draft_tokens + lo + i);
    const int row = !draft ? 0 : a.draft_rows ? __ldg(a.draft_rows + lo + i) : lo + i;
    const float u = __ldg(a.u_accept + lo + i);
    if (parent < -1 || parent >= i || x < 0 || x >= a.V || !(u >= 0.f && u < 1.f) || row < 0 ||
        (draft && row >= a.draft_rows_count)) {
      bad = true;
      continue;
    }
    const float p = load_prob(target + (row0 + parent + 1) * a.target_stride + x);
    const float q = draft ? load_prob(draft + row * a.draft_stride + x) : 1.f;
    const int first = atomicCAS(&sh.of_parent[parent + 1], -1, row);
    bad |= bad_prob(p) || bad_prob(q) || (first != -1 && first != row);
    sh.parent[i] = (short)parent;
    sh.x[i] = x;
    sh.row[i] = row;
    sh.u[i] = u;
    sh.p[i] = p;
    sh.q[i] = q;
    // both factors have 24 bits, so the 64-bit product is exact
    sh.as_first[i] = (double)u * (double)q < (double)p;
  }
  if (bad) atomicOr(&sh.bad, 1);
  __syncthreads();
  bad = sh.bad;
  cluster.barrier_wait();

  W w{};
  int passes = 0;
  uint32_t* const holes = reinterpret_cast<uint32_t*>(marks + marks_words<P, C>(a.V));
  // Sums the weights w over the cluster.  All CTAs take part, and all learn of bad probabilities.
  auto sum = [&]() {
    const Share<C> at(w.vectors(), rank);
    const int w0 = min(at.end, at.begin + warp * at.part), w1 = min(at.end, w0 + at.part);
    Range range;
    const int64_t mine = warp_total(w.sum_range(w0, w1, &range, marks + tid));
    const bool odd = __any_sync(~0u, range.bad());
    if (lane == 0) {
      sh.warp_sum[warp] = mine;
      if (odd) atomicOr(&sh.odd, 1);
    }
    __syncthreads();
    const int turn = passes & 1;
    if (tid < C) {
      int64_t slice = 0;
      for (int i = 0; i < kWarps; ++i) slice += sh.warp_sum[i];
      Shared* other = cluster.map_shared_rank(&sh, tid);
      other->slice_sum[turn][rank] = slice;
      other->slice_bad[turn][rank] = sh.odd;
    }
    cluster.sync();
    ++passes;
    int64_t total = 0;
    for (int i = 0; i < C; ++i) {
      total += sh.slice_sum[turn][i];
      bad |= sh.slice_bad[turn][i] != 0;
    }
    return total;
  };

  // The walk, by the first warp of each CTA of the cluster, up to the next sum that it needs.
  while (!bad) {
    if (warp == 0) {
      __syncwarp();
      // the last accepted token, how many, refused children of it
      int node = sh.step.node, acc = sh.step.acc, refused = sh.step.refused, at_token = sh.walk.at;
      float share = sh.walk.s, taken = sh.walk.c;  // s and c
      int64_t removed = sh.walk.removed;           // without a draft: P of the refused ids
      // the first token after i whose parent is `node`, or n
      auto next_child = [&](int i) {
        for (int base = (i + 1) & ~31; base < n; base += 32) {
          const int j = base + lane;
          const unsigned m = __ballot_sync(~0u, j > i && j < n && sh.parent[min(j, n - 1)] == node);
          if (m) return base + __ffs(m) - 1;
        }
        return n;
      };
      // Whether token i is accepted with share s; for a draft with probabilities.
      auto accepts = [&](int i, float s) {
        if (!refused) return (bool)sh.as_first[i];
        const float p = sh.p[i], q = sh.q[i], cut = q * taken;
        const double left = p > cut ? (double)(mass_at(p) - mass_at(cut)) * 9.094947017729282379150390625e-13 : 0.0;
        return (double)sh.u[i] * (double)(q * s) < left;
      };
      auto accept = [&](int i) {
        if (lane == 0) sh.path[acc] = (short)i;
        ++acc;
        node = i;
        refused = 0;
        share = 1.f;
        taken = 0.f;
        removed = 0;
      };
      auto walk = [&]() {  // true: a sum is needed
        while (true) {
          const int i = acc < a.max_path ? next_child(at_token) : n;
          if (i >= n) return false;
          at_token = i;
          if (draft) {
            if (accepts(i, share)) {
              accept(i);
              continue;
            }
            ++refused;
            taken += share;
            if (share == 0.f) continue;  // nothing is left, and nothing will be
            // the next one, should it be accepted with a share that can only be too large
            const int next = next_child(i);
            if (next >= n || !accepts(next, share)) return true;
            at_token = next;
            accept(next);
          } else {
            bool again = false;  // a refused child of the same parent has the same id
            if (refused) {
              const int x = sh.x[i];
              for (int base = 0; base < i && !again; base += 32) {
                const int j = min(base + lane, n - 1);
                again = __any_sync(~0u, base + lane < i && sh.parent[j] == node && sh.x[j] == x);
              }
            }
            const float p = sh.p[i];
            const bool ok = !again && (refused ? (double)sh.u[i] * (double)share < (double)p : (bool)sh.as_first[i]);
            if (ok) {
              accept(i);
              continue;
            }
            ++refused;
            if (!again) removed += mass_at(p);
            share = share_of(max(((int64_t)1 << 40) - removed, (int64_t)0));
          }
        }
      };
      const bool more = walk();
      __syncwarp();
      if (lane == 0) {
        sh.step = {node, acc, refused, refused && draft ? sh.row[at_token] : 0, taken, !more};
        sh.walk = {at_token, share, taken, removed};
      }
    }
    __syncthreads();
    if (sh.step.end) break;
    w.set(target + (row0 + sh.step.node + 1) * a.target_stride, draft + sh.step.row * a.draft_stride, -1, a.V);
    w.taken = sh.step.taken;
    const int64_t total = sum();
    if (tid == 0) {
      sh.total = total;
      sh.walk.s = fminf(share_of(total), 1.f);
    }
  }
  const int node = sh.step.node, acc = sh.step.acc, refused = sh.step.refused;

  int64_t total = 0;
  if (!bad) {  // uniform over the cluster
    total = sh.total;
    if (!draft || !refused) {  // else the last sum is that of what is left
      w.set(target + (row0 + node + 1) * a.target_stride, nullptr, -1, a.V);
      w.holes = nullptr;
      if (refused) {  // a certain draft's
        const int slice = (w.vectors() + C - 1) / C;
        w.hole_base = rank * slice;
        for (int i = tid; i < (slice * N + 31) / 32; i += kThreads) holes[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
          const int e = sh.x[i] + w.a - w.hole_base * N;
          if (sh.parent[i] == node && e >= 0 && e < slice * N) atomicOr(&holes[e >> 5], 1u << (e & 31));
        }
        __syncthreads();
        w.holes = holes;
      }
      total = sum();
    }
    if (!bad && total == 0 && refused) {  // nothing is left: draw from p itself
      w.set(w.p, nullptr, -1, a.V);
      w.holes = nullptr;
      total = sum();
    }
    bad |= total == 0;
  }

  int32_t* out = a.tokens + (int64_t)b * a.token_stride;
  if (rank == 0) {
    int32_t* path = a.path ? a.path + (int64_t)b * a.path_stride : nullptr;
    for (int i = tid; i <= a.max_path; i += kThreads) {
      const int node_at = !bad && i < acc ? sh.path[i] : -1;
      if (bad || i != acc) out[i] = node_at >= 0 ? sh.x[node_at] : -1;
      if (path && i < a.max_path) path[i] = node_at;
    }
    if (tid == 0) {
      if (a.accepted) a.accepted[b] = bad ? 0 : acc;
      if (a.row_status) a.row_status[b] = bad ? CLSAMPLE_ROW_INVALID : CLSAMPLE_ROW_OK;
    }
  }
  if (bad) return;
  // floor(u31 total / 2^31) with total below 2^58
  const int64_t u31 = __float2ll_rz(u_last * 2147483648.f);
  int64_t left = u31 * (total >> 31) + ((u31 * (total & 0x7fffffff)) >> 31);
  const int64_t* const slices = sh.slice_sum[(passes - 1) & 1];
  for (int i = 0; i < rank; ++i) left -= slices[i];
  if (left < 0 || left >= slices[rank]) return;  // another slice's
  const Share<C> at(w.vectors(), rank);
  int part = 0;  // the warp whose part holds the threshold
  while (left >= sh.warp_sum[part]) left -= sh.warp_sum[part++];
  // the batch of that warp: lane i adds up batch i
  int p0 = at.begin + part * at.part;
  const int p1 = min(at.end, p0 + at.part);
  const int batches = (p1 - p0 + kBatch - 1) / kBatch;  // at most 32
  int64_t run = 0;
  if (lane < batches)
#pragma unroll 8
    for (int i = 0; i < 32; ++i) run += marks[lane * kThreads + part * 32 + (i + lane) % 32];
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
int smem_bytes(int V) {
  constexpr int N = 16 / sizeof(P);
  const int vectors = (V + 2 * N - 2) / N, share = (vectors + C - 1) / C;
  return marks_bytes<P, C>(V) + (share * N + 31) / 32 * (int)sizeof(uint32_t);
}

template <class P, int C>
cudaError_t launch_tree(const clsample_verify_tree_args_t& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.B * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem_bytes<P, C>(a.V);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  static std::atomic<uint64_t> allowed;
  cudaError_t e = allow_smem_once(verify_tree_kernel<P, C>, smem_bytes<P, C>(kMaxVocab), &allowed);
  if (C > 8 && e == cudaSuccess) {
    static std::atomic<uint64_t> large;
    e = allow_once(verify_tree_kernel<P, C>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1, &large);
  }
  return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, verify_tree_kernel<P, C>, a) : e;
}

// As for clsample_verify: the largest cluster with which all requests would be resident at once with four CTAs
// a multiprocessor, which is what registers allow.  (Shared memory does not in all cases: with arrays for 1023
// tokens and bits for refused ids, float32 and clusters of two, a CTA has 60 KB over 151936 tokens and 81 over
// 262144, so three or two fit, and of 229 requests and more some begin when others have ended; with clusters of four
// over 262144 three fit.)  One request of 6 refusals over 151936 tokens: 29 us on 16 CTAs, 40 on 8.  (On an earlier version 64 requests
// on 16 CTAs each, not all resident: 47 us instead of 51 where one of them has far more refusals than the
// others, but 110 instead of 82 where all have 6; now 48 and 77 on 8.  Three CTAs a multiprocessor of 80
// registers, not all resident either: 41 and 98.)
template <class P>
cudaError_t launch_tree(const clsample_verify_tree_args_t& a, int sms, cudaStream_t st) {
  const int64_t slots = (int64_t)sms * kCtasPerSm;
  if (a.B * (int64_t)16 <= slots) return launch_tree<P, 16>(a, st);
  if (a.B * (int64_t)8 <= slots) return launch_tree<P, 8>(a, st);
  if (a.B * (int64_t)4 <= slots) return launch_tree<P, 4>(a, st);
  return launch_tree<P, 2>(a, st);
}

}  // namespace
}  // namespace clsample

extern "C" int clsample_verify_tree(const clsample_verify_tree_args_t* a, clsample_stream_t stream) {
  using namespace clsample;
  if (!a) return CLSAMPLE_ERR_NULL;
  if (a->B < 0 || a->B > (1 << 24) - 1 || a->N < 0) return CLSAMPLE_ERR_BATCH;
  if (a->V <= 0 || a->V > kMaxVocab) return CLSAMPLE_ERR_VOCAB;
  if (a->dtype != CLSAMPLE_LOGITS_F32 && a->dtype != CLSAMPLE_LOGITS_BF16) return CLSAMPLE_ERR_DTYPE;
  if (a->max_draft < 0 || a->max_draft > kMaxNodes || a->max_path < 0 || a->max_path > a->max_draft ||
      a->draft_rows_count < 0)
    return CLSAMPLE_ERR_SHAPE;
  if (a->target_stride < a->V || (a->draft && a->draft_stride < a->V) || a->token_stride <= a->max_path ||
      (a->path && a->path_stride < a->max_path))
    return CLSAMPLE_ERR_STRIDE;
  if (a->B == 0) return CLSAMPLE_SUCCESS;
  if (!a->target || !a->cu_draft || !a->u_sample || !a->tokens ||
      (a->N > 0 && (!a->draft_tokens || !a->u_accept || !a->parents)))
    return CLSAMPLE_ERR_NULL;
  int sms = 0;
  const int rc = check_device(nullptr, &sms);
  if (rc != CLSAMPLE_SUCCESS) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      a->dtype == CLSAMPLE_LOGITS_F32 ? launch_tree<float>(*a, sms, st) : launch_tree<__nv_bfloat16>(*a, sms, st);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? CLSAMPLE_SUCCESS : CLSAMPLE_ERR_CUDA;
}
