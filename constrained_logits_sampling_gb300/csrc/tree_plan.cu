// clsample_tree_plan: what each row of a tree may see, and where it stands (include/clsample.h).
//
// One CTA per request, a thread for each word of each row: it walks from the row to the root over
// parents in shared memory and sets the bits that fall into its word; parents come before their
// children, so it may stop below the word.  All of it is latency: one load of the parents, then as many
// steps in shared memory as the tree is deep.
#include "paged.cuh"

namespace clsample {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 1024;

__global__ void __launch_bounds__(kThreads) tree_plan_kernel(const __grid_constant__ clsample_tree_plan_args_t a) {
  __shared__ short up[kMaxRows];  // a row's parent among the request's rows; the root's is -1
  const int b = blockIdx.x, tid = threadIdx.x;
  const int lo = __ldg(a.cu_draft + b), hi = __ldg(a.cu_draft + b + 1), len = __ldg(a.kv_lens + b);
  if (a.cu_new && tid == 0) {
    a.cu_new[b] = (int)((unsigned)lo + (unsigned)b);
    if (b == a.B - 1) a.cu_new[a.B] = (int)((unsigned)hi + (unsigned)a.B);
  }
  const bool placed = lo >= 0 && hi >= lo && hi <= a.N;
  const int n = hi - lo;
  bool bad = !placed || n > a.max_draft || len <= n || len > kMaxLen;
  if (!bad) {
    for (int i = tid; i < n; i += kThreads) {
      const int p = __ldg(a.parents + lo + i);
      bad |= p < -1 || p >= i;
      up[i + 1] = (short)(p + 1);
    }
    if (tid == 0) up[0] = -1;
  }
  bad = __syncthreads_or(bad);
  if (a.row_status && tid == 0) a.row_status[b] = bad ? CLSAMPLE_ROW_INVALID : CLSAMPLE_ROW_OK;
  if (!placed) return;
  const int64_t row0 = (int64_t)lo + b;
  const int words = (a.max_draft + 32) / 32;
  const int64_t items = ((int64_t)n + 1) * words;
  for (int64_t it = tid; it < items; it += kThreads) {
    const int64_t r = it / words;
    const int w = (int)(it - r * words);
    uint32_t bits = 0;
    int steps = -1;
    if (!bad)
      for (int at = (int)r; at >= (w == 0 ? 0 : 32 * w); at = up[at]) {
        ++steps;
        if ((at >> 5) == w && (a.window <= 0 || steps < a.window)) bits |= 1u << (at & 31);
      }
    a.mask[(row0 + r) * a.mask_stride + w] = bits;
    if (w == 0 && a.positions) a.positions[row0 + r] = bad ? 0 : len - n - 1 + steps;
  }
}

}  // namespace
}  // namespace clsample

extern "C" int clsample_tree_plan(const clsample_tree_plan_args_t* a, clsample_stream_t stream) {
  using namespace clsample;
  if (!a) return CLSAMPLE_ERR_NULL;
  if (a->B < 0 || a->B > (1 << 24) - 1 || a->N < 0) return CLSAMPLE_ERR_BATCH;
  if (a->max_draft < 0 || a->max_draft >= kMaxRows || a->window < 0) return CLSAMPLE_ERR_SHAPE;
  if (a->mask_stride < (a->max_draft + 32) / 32) return CLSAMPLE_ERR_STRIDE;
  if (a->B == 0) return CLSAMPLE_SUCCESS;
  if (!a->cu_draft || !a->kv_lens || !a->mask || (a->N > 0 && !a->parents)) return CLSAMPLE_ERR_NULL;
  const int rc = check_device();
  if (rc != CLSAMPLE_SUCCESS) return rc;
  tree_plan_kernel<<<a->B, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(*a);
  return cudaGetLastError() == cudaSuccess ? CLSAMPLE_SUCCESS : CLSAMPLE_ERR_CUDA;
}
