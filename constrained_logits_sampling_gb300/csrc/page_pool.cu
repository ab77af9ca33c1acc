// clsample_pages_fork, _reserve and _trim: which sequence holds which page of a cache (rules in
// include/clsample.h).
//
// Counting references needs no order, and free pages are a set of bits, so whatever order
// atomics take, the state after a call is the same.  What has an order, the giving out of free
// pages, is one CTA's work: it needs a prefix sum over the sequences and one over the bits.  All of it is
// latency: a few dependent loads and barriers.
#include "paged.cuh"

namespace clsample {
namespace {

constexpr int kThreads = 256;
constexpr int kReserveThreads = 1024;

struct PoolParams {
  clsample_page_pool_t pool;
  clsample_page_batch_t batch;
};

__device__ __forceinline__ bool valid_page(const clsample_page_pool_t& pool, int id) {
  return id >= 0 && id < pool.num_pages;
}
__device__ __forceinline__ int pages_of(int len, int page_size) { return len / page_size + (len % page_size != 0); }

// One CTA a pair.  A pair that is done has a dst that no other pair names, so nobody reads what it writes.
__global__ void __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ PoolParams P, const int32_t* src_of,
                                                        const int32_t* dst_of, int n, int32_t* status) {
  const clsample_page_pool_t& pool = P.pool;
  const clsample_page_batch_t& q = P.batch;
  const int i = blockIdx.x, tid = threadIdx.x;
  const int src = __ldg(src_of + i), dst = __ldg(dst_of + i);
  int bad = src < 0 || src >= q.B || dst < 0 || dst >= q.B;
  for (int k = tid; k < n; k += kThreads) bad |= __ldg(src_of + k) == dst || (k != i && __ldg(dst_of + k) == dst);
  bad = __syncthreads_or(bad);
  int len = 0, need = 0;
  if (!bad) {  // (src is no dst and dst is this pair's: neither changes meanwhile)
    len = q.kv_lens[src];
    const int held = q.held[src];
    bad = len < 0 || len > capacity_of(q.max_pages, pool.page_size) || held > q.max_pages || q.held[dst] != 0;
    need = bad ? 0 : pages_of(len, pool.page_size);
    bad |= need > held;
  }
  const int32_t* row = q.page_table + src * q.table_stride;
  if (!bad)
    for (int k = tid; k < need; k += kThreads) {
      const int id = row[k];
      // (counts may grow meanwhile, from 1 at least)
      bad |= !valid_page(pool, id) || __ldcg(pool.refs + id) < 1;
    }
  bad = __syncthreads_or(bad);
  if (!bad) {
    int32_t* to = q.page_table + dst * q.table_stride;
    for (int k = tid; k < need; k += kThreads) {
      const int id = row[k];
      to[k] = id;
      atomicAdd(pool.refs + id, 1);
    }
    if (tid == 0) {
      q.held[dst] = need;
      q.kv_lens[dst] = len;
    }
  }
  if (status && tid == 0) status[i] = bad ? CLSAMPLE_ROW_INVALID : CLSAMPLE_ROW_OK;
}

// One CTA a sequence.
__global__ void __launch_bounds__(kThreads) trim_kernel(const __grid_constant__ PoolParams P, int32_t* status) {
  const clsample_page_pool_t& pool = P.pool;
  const clsample_page_batch_t& q = P.batch;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int len = q.kv_lens[b], held = q.held[b];
  bool bad = len < 0 || len > capacity_of(q.max_pages, pool.page_size) || held < 0 || held > q.max_pages;
  const int keep = bad ? 0 : pages_of(len, pool.page_size);
  bad |= keep > held;
  const bool can = !bad;
  if (can) {
    int32_t* row = q.page_table + b * q.table_stride;
    for (int k = keep + tid; k < held; k += kThreads) {
      const int id = row[k];
      row[k] = -1;
      if (!valid_page(pool, id)) {
        bad = true;
        continue;
      }
      const int was = atomicSub(pool.refs + id, 1);
      if (was == 1) {
        atomicOr(pool.free_bits + (id >> 5), 1u << (id & 31));
      } else if (was < 1) {  // nobody held it
        atomicAdd(pool.refs + id, 1);
        bad = true;
      }
    }
  }
  const bool any = __syncthreads_or(bad);  // and all have read held[b]
  if (tid == 0) {
    if (can) q.held[b] = keep;
    if (status) status[b] = any ? CLSAMPLE_ROW_INVALID : CLSAMPLE_ROW_OK;
  }
}

// Sum over the block and each thread's exclusive prefix.
template <class T>
__device__ __forceinline__ T block_prefix(T v, T* buf, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T run = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T up = __shfl_up_sync(~0u, run, o);
    if (lane >= o) run += up;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = run;
  __syncthreads();
  T w = buf[lane];  // 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T up = __shfl_up_sync(~0u, w, o);
    if (lane >= o) w += up;
  }
  const T base = __shfl_sync(~0u, w, warp) - buf[warp];
  *total = __shfl_sync(~0u, w, 31);
  return base + run - v;
}

// What a sequence is about to write: `count` tokens behind `len`, to the pages first .. last of its
// row, of which it holds those before `held`.
struct Writes {
  int len, count, held, first, last;
};

// One CTA, a thread a sequence.  A page that sequences of the call would write to, where any of
// them is shared: each takes its reference back first, and if none is left nobody else holds it; the last
// of them, by a maximum over stamps, then keeps it.  Stamps carry the call's number, so they need not be
// cleared.  Without a shared page none of that is done (7.3 us to 4.3 for 240 sequences).
// Of up to 1024 sequences, a thread keeps what it has read of its one; beyond that copies tells it from
// one pass to the next whether it is INVALID (-2), where its pages start in the list and how many it needs.
__global__ void __launch_bounds__(kReserveThreads) reserve_kernel(const __grid_constant__ PoolParams P,
                                                                  const int32_t* new_tokens, int32_t* copies,
                                                                  int32_t* status, int32_t* free_pages) {
  const clsample_page_pool_t& pool = P.pool;
  const clsample_page_batch_t& q = P.batch;
  constexpr int kAlone = 8;  // pages that a thread hands out by itself
  struct Long { int b, from, count, at; };
  __shared__ int64_t wide_buf[32];
  __shared__ int buf[32], near[kReserveThreads];  // near: the first pages of the list
  __shared__ Long longs[kReserveThreads];
  __shared__ int long_count;
  const int tid = threadIdx.x, page = pool.page_size, cap = capacity_of(q.max_pages, page);
  const bool one = q.B <= kReserveThreads;
  const uint32_t number = *pool.epoch + 1;  // the call's
  const uint64_t call = (uint64_t)max(number, 1u) << 32;
  // free pages: each thread counts a run of the words
  const int words = (pool.num_pages + 31) / 32, each = (words + kReserveThreads - 1) / kReserveThreads;
  const int w0 = min(words, tid * each), w1 = min(words, w0 + each);
  uint32_t first_word = 0;
  int mine = 0, available;
#pragma unroll 4
  for (int i = w0; i < w1; ++i) {
    const uint32_t bits = pool.free_bits[i];
    if (i == w0) first_word = bits;
    mine += __popc(bits);
  }
  auto load = [&](int b) {
    Writes w{q.kv_lens[b], __ldg(new_tokens + b), q.held[b], 0, -1};
    if (w.count > 0) {
      w.first = w.len / page;
      w.last = (int)(((int64_t)w.len + w.count - 1) / page);
    }
    return w;
  };
  auto own_last = [](const Writes& w) { return min(w.last, w.held - 1); };
  // whether sequence b keeps page id, which it would write to
  bool shares = false;  // uniform, below: a page to write to is held by several
  auto keeps = [&](int b, int id) {
    return !shares ||
           (__ldcg(pool.refs + id) == 0 && __ldcg(pool.stamps + id) == (call | (unsigned)(b + 1)));
  };
  Writes mine_w{0, 0, 0, 0, -1};  // of sequence tid
  bool mine_bad = false;
  int mine_id = 0;                // the first page that it writes to, if it holds that
  auto writes_of = [&](int b) { return one ? mine_w : load(b); };
  auto page_at = [&](int b, const Writes& w, int k) {
    return one && k == w.first ? mine_id : q.page_table[b * q.table_stride + k];
  };
  auto is_bad = [&](int b) { return one ? mine_bad : copies[3 * (int64_t)b] == -2; };

  for (int b = tid; b < q.B; b += kReserveThreads) {
    const Writes w = load(b);
    bool bad = w.len < 0 || w.count < 0 || w.len > cap || w.count > cap - w.len || w.held < 0 || w.held > q.max_pages ||
               pages_of(w.len, page) > w.held;
    if (!bad)
      for (int k = w.first; k <= own_last(w); ++k) {
        const int id = q.page_table[b * q.table_stride + k];
        if (k == w.first) mine_id = id;
        const int refs = valid_page(pool, id) ? __ldcg(pool.refs + id) : 0;
        bad |= refs < 1;
        shares |= refs > 1;
      }
    if (!one) copies[3 * (int64_t)b] = bad ? -2 : -1;
    mine_w = w;
    mine_bad = bad;
  }
  int rank = block_prefix(mine, buf, &available);
  shares = __syncthreads_or(shares);
  if (number == 0) {  // where 32 bits end stamps start anew, as those of earlier calls would be larger
    for (int i = tid; i < pool.num_pages; i += kReserveThreads) pool.stamps[i] = 0;
    __syncthreads();
  }
  if (shares) {
    for (int b = tid; b < q.B; b += kReserveThreads) {
      if (is_bad(b)) continue;
      const Writes w = writes_of(b);
      for (int k = w.first; k <= own_last(w); ++k) {
        const int id = page_at(b, w, k);
        atomicSub(pool.refs + id, 1);
        atomicMax(reinterpret_cast<unsigned long long*>(pool.stamps + id),
                  (unsigned long long)(call | (unsigned)(b + 1)));
      }
    }
    __syncthreads();
  }

  int64_t total = 0;
  int mine_at = 0, mine_need = 0;
  for (int base = 0; base < q.B; base += kReserveThreads) {  // uniform
    const int b = base + tid;
    int need = 0;
    int64_t sum;
    if (b < q.B && !is_bad(b)) {
      const Writes w = writes_of(b);
      if (shares)
        for (int k = w.first; k <= own_last(w); ++k) need += !keeps(b, page_at(b, w, k));
      need += max(0, w.last + 1 - max(w.held, w.first));
    }
    // sequences may lack 2^30 pages each; where the table has no room for that 32 bits do (a reservation for one
    // prompt's sequences 4.3 us, 4.5 in 64 bits)
    int64_t before;
    if (q.max_pages > kMaxLen / kReserveThreads) {
      before = block_prefix((int64_t)need, wide_buf, &sum);
    } else {
      int narrow_sum;
      before = block_prefix(need, buf, &narrow_sum);
      sum = narrow_sum;
    }
    mine_at = (int)min(total + before, (int64_t)0x7fffffff);
    mine_need = need;
    if (b < q.B && !one) {
      copies[3 * (int64_t)b + 1] = mine_at;
      copies[3 * (int64_t)b + 2] = need;
    }
    total += sum;
  }
  const bool enough = total <= available;
  if (enough)
    for (int i = w0; i < w1 && rank < total; ++i) {
      uint32_t bits = i == w0 ? first_word : pool.free_bits[i];
      while (bits && rank < total) {
        const int id = i * 32 + __ffs(bits) - 1;
        if (rank < kReserveThreads) near[rank] = id;
        else pool.list[rank] = id;
        ++rank;
        bits &= bits - 1;
      }
      pool.free_bits[i] = bits;
    }
  if (tid == 0) long_count = 0;
  __syncthreads();
  auto listed = [&](int at) { return at < kReserveThreads ? near[at] : pool.list[at]; };

  for (int base = 0; base < q.B; base += kReserveThreads) {
    const int b = base + tid;
    if (b < q.B) {
      int32_t* copy = copies + 3 * (int64_t)b;
      const bool bad = is_bad(b);
      int at = one ? mine_at : copy[1];
      const int need = one ? mine_need : copy[2];
      int from = -1, to = -1, slots = 0;
      if (!bad) {
        const Writes w = writes_of(b);
        int32_t* row = q.page_table + b * q.table_stride;
        if (shares)
          for (int k = w.first; k <= own_last(w); ++k) {
            const int id = page_at(b, w, k);
            if (!enough) {
              atomicAdd(pool.refs + id, 1);
            } else if (keeps(b, id)) {
              atomicExch(pool.refs + id, 1);
            } else {
              const int page_id = listed(at++);
              row[k] = page_id;
              pool.refs[page_id] = 1;
              if (k == w.first && w.len % page) {
                from = id;
                to = page_id;
                slots = w.len % page;
              }
            }
          }
        const int fresh = max(w.held, w.first), lacks = w.last + 1 - fresh;
        if (enough && lacks > 0) {
          if (lacks > kAlone) {
            longs[atomicAdd(&long_count, 1)] = Long{b, fresh, lacks, at};
          } else {
            for (int k = 0; k < lacks; ++k) {
              const int page_id = listed(at + k);
              row[fresh + k] = page_id;
              pool.refs[page_id] = 1;
            }
          }
          q.held[b] = w.last + 1;
        }
      }
      copy[0] = from;
      copy[1] = to;
      copy[2] = slots;
      if (status)
        status[b] = bad ? CLSAMPLE_ROW_INVALID : !enough && need > 0 ? CLSAMPLE_ROW_OVERFLOW : CLSAMPLE_ROW_OK;
    }
    __syncthreads();
    const int todo = long_count;
    for (int i = 0; i < todo; ++i) {
      const Long l = longs[i];
      for (int k = tid; k < l.count; k += kReserveThreads) {
        const int page_id = listed(l.at + k);
        q.page_table[l.b * q.table_stride + l.from + k] = page_id;
        pool.refs[page_id] = 1;
      }
    }
    if (one) break;
    __syncthreads();
    if (tid == 0) long_count = 0;
    __syncthreads();
  }
  if (tid == 0) {
    *pool.epoch = (uint32_t)(call >> 32);
    if (free_pages) *free_pages = available - (enough ? (int)total : 0);
  }
}

int check_pool(const clsample_page_pool_t* pool, const clsample_page_batch_t* batch) {
  if (!pool || !batch) return CLSAMPLE_ERR_NULL;
  if (batch->B < 0 || batch->B > (1 << 24) - 1) return CLSAMPLE_ERR_BATCH;
  if (pool->num_pages < 0 || pool->num_pages > kMaxLen || pool->page_size < 1 || batch->max_pages < 0)
    return CLSAMPLE_ERR_SHAPE;
  if (batch->table_stride < batch->max_pages) return CLSAMPLE_ERR_STRIDE;
  if (batch->B == 0) return CLSAMPLE_SUCCESS;
  if (!batch->held || !batch->kv_lens || (!batch->page_table && batch->max_pages > 0) || !pool->epoch ||
      (pool->num_pages > 0 && (!pool->refs || !pool->free_bits || !pool->stamps || !pool->list)))
    return CLSAMPLE_ERR_NULL;
  return CLSAMPLE_SUCCESS;
}

}  // namespace
}  // namespace clsample

extern "C" {

int clsample_pages_fork(const clsample_page_pool_t* pool, const clsample_page_batch_t* batch, const int32_t* src,
                        const int32_t* dst, int32_t n, int32_t* status, clsample_stream_t stream) {
  using namespace clsample;
  int rc = check_pool(pool, batch);
  if (rc != CLSAMPLE_SUCCESS) return rc;
  if (n < 0 || n > (1 << 24) - 1) return CLSAMPLE_ERR_BATCH;
  if (n == 0) return CLSAMPLE_SUCCESS;
  if (!src || !dst) return CLSAMPLE_ERR_NULL;
  if ((rc = check_device()) != CLSAMPLE_SUCCESS) return rc;
  fork_kernel<<<n, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(PoolParams{*pool, *batch}, src, dst, n, status);
  return cudaGetLastError() == cudaSuccess ? CLSAMPLE_SUCCESS : CLSAMPLE_ERR_CUDA;
}

int clsample_pages_reserve(const clsample_page_pool_t* pool, const clsample_page_batch_t* batch,
                           const int32_t* new_tokens, int32_t* copies, int32_t* row_status, int32_t* free_pages,
                           clsample_stream_t stream) {
  using namespace clsample;
  int rc = check_pool(pool, batch);
  if (rc != CLSAMPLE_SUCCESS) return rc;
  if (batch->B == 0) return CLSAMPLE_SUCCESS;
  if (!new_tokens || !copies) return CLSAMPLE_ERR_NULL;
  if ((rc = check_device()) != CLSAMPLE_SUCCESS) return rc;
  reserve_kernel<<<1, kReserveThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      PoolParams{*pool, *batch}, new_tokens, copies, row_status, free_pages);
  return cudaGetLastError() == cudaSuccess ? CLSAMPLE_SUCCESS : CLSAMPLE_ERR_CUDA;
}

int clsample_pages_trim(const clsample_page_pool_t* pool, const clsample_page_batch_t* batch, int32_t* row_status,
                        clsample_stream_t stream) {
  using namespace clsample;
  int rc = check_pool(pool, batch);
  if (rc != CLSAMPLE_SUCCESS) return rc;
  if (batch->B == 0) return CLSAMPLE_SUCCESS;
  if ((rc = check_device()) != CLSAMPLE_SUCCESS) return rc;
  trim_kernel<<<batch->B, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(PoolParams{*pool, *batch}, row_status);
  return cudaGetLastError() == cudaSuccess ? CLSAMPLE_SUCCESS : CLSAMPLE_ERR_CUDA;
}

}  // extern "C"
