// clsample_keep_path and clsample_copy_pages: keys and values moved within a paged cache, in all of
// its layers (rules in include/clsample.h).  Both are bound by memory: what is moved is read once and
// written once, in pieces of 16 bytes where addresses, strides and heads allow it, of 8, 4 or 2 otherwise.
#include "paged.cuh"

namespace clsample {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPath = 1023;

template <int kBytes> struct Piece;
template <> struct Piece<16> { using T = uint4; };
template <> struct Piece<8> { using T = uint2; };
template <> struct Piece<4> { using T = uint32_t; };
template <> struct Piece<2> { using T = uint16_t; };

// The cache in pieces.
struct CacheShape {
  int64_t layer, page, slot, head;  // strides
  int per_head;                     // pieces of a head
};

// A thread has one column (a place of a head, in one layer, of keys or of values) of one request
// and moves it through all places of the path in turn.  A place is written when all that is read from it
// has been read, as numbers of a path only grow: nothing is staged, and no thread waits for another.
template <int kBytes>
__global__ void __launch_bounds__(kThreads) keep_path_kernel(const __grid_constant__ clsample_keep_path_args_t a,
                                                             const __grid_constant__ CacheShape c, int parts) {
  using T = typename Piece<kBytes>::T;
  constexpr int kAhead = 8;  // pieces of a thread in flight
  __shared__ int64_t from[kMaxPath + 1], to[kMaxPath + 1];
  __shared__ int stays;  // tokens that are in their places: the first ones
  const int b = blockIdx.x / parts, part = blockIdx.x % parts, tid = threadIdx.x;
  const int lo = __ldg(a.cu_draft + b), hi = __ldg(a.cu_draft + b + 1), len = __ldg(a.kv_lens + b);
  const int count = __ldg(a.accepted + b), n = hi - lo;
  bool bad = lo < 0 || hi < lo || hi > a.N || len <= n || len > capacity_of(a.max_pages, a.page_size) || count < 0 ||
             count > min(n, a.max_path);
  const int first = len - n;  // the first place of the path
  if (tid == 0) stays = 0;
  __syncthreads();
  if (!bad) {
    const int32_t* path = a.path + (int64_t)b * a.path_stride;
    const int32_t* table = a.page_table + (int64_t)b * a.table_stride;
    for (int i = tid; i < count; i += kThreads) {
      const int x = __ldg(path + i), before = i ? __ldg(path + i - 1) : -1;
      if (x <= before || x >= n) {
        bad = true;
      } else if (x == i) {
        atomicAdd(&stays, 1);
      } else {
        const int src = first + x, dst = first + i;
        const int src_page = __ldg(table + src / a.page_size), dst_page = __ldg(table + dst / a.page_size);
        bad |= src_page < 0 || src_page >= a.num_pages || dst_page < 0 || dst_page >= a.num_pages;
        from[i] = src_page * c.page + src % a.page_size * c.slot;
        to[i] = dst_page * c.page + dst % a.page_size * c.slot;
      }
    }
  }
  bad = __syncthreads_or(bad);
  if (part == 0 && tid == 0) {
    a.new_lens[b] = bad ? len : first + count;
    if (a.row_status) a.row_status[b] = bad ? CLSAMPLE_ROW_INVALID : CLSAMPLE_ROW_OK;
  }
  if (bad) return;
  const int begin = stays;
  if (begin >= count) return;
  // (below 2^31; a step is about half of them, so the first column past them needs 32 bits)
  const unsigned heads = (unsigned)(c.per_head * a.Hkv), columns = 2 * a.layers * heads;
  for (unsigned col = part * kThreads + tid; col < columns; col += (unsigned)parts * kThreads) {
    const int plane = (int)(col / heads), rest = (int)(col % heads);  // planes: keys of all layers, then values
    const int layer = plane < a.layers ? plane : plane - a.layers;
    T* at = reinterpret_cast<T*>(plane < a.layers ? a.k_cache : a.v_cache) + layer * c.layer +
            rest / c.per_head * c.head + rest % c.per_head;
    for (int i0 = begin; i0 < count; i0 += kAhead) {
      T x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i0 + k < count) x[k] = at[from[i0 + k]];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i0 + k < count) at[to[i0 + k]] = x[k];
    }
  }
}

// An item is a share of one copy's pieces in one plane (keys or values of a layer).  A CTA takes several
// where there are many, as most copies of a call may be none (3840 CTAs of nothing took 7.4 us).
template <int kBytes>
__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const __grid_constant__ clsample_copy_pages_args_t a,
                                                              const __grid_constant__ CacheShape c, int parts) {
  using T = typename Piece<kBytes>::T;
  constexpr int kAhead = 8;  // pieces of a thread in flight
  const int planes = 2 * a.layers, per_copy = planes * parts;
  const int64_t items = (int64_t)a.n * per_copy;
  const int heads = c.per_head * a.Hkv, step = parts * kThreads, step_slots = step / heads, step_rest = step % heads;
  const bool flat = c.head == c.per_head;  // a slot's heads lie side by side
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int i = (int)(item / per_copy), rest = (int)(item - (int64_t)i * per_copy);
    const int plane = rest / parts, part = rest % parts;
    const int from = __ldg(a.copies + 3 * (int64_t)i), to = __ldg(a.copies + 3 * (int64_t)i + 1),
              slots = __ldg(a.copies + 3 * (int64_t)i + 2);
    const bool none = from < 0 || slots == 0;
    const bool bad = !none && (from >= a.num_pages || to < 0 || to >= a.num_pages || slots < 0 || slots > a.page_size);
    if (a.status && rest == 0 && threadIdx.x == 0) a.status[i] = bad ? CLSAMPLE_ROW_INVALID : CLSAMPLE_ROW_OK;
    if (none || bad || from == to) continue;
    const int layer = plane < a.layers ? plane : plane - a.layers;
    T* at = reinterpret_cast<T*>(plane < a.layers ? a.k_cache : a.v_cache) + layer * c.layer;
    const T* src = at + from * c.page;
    T* dst = at + to * c.page;
    // this thread's place (a slot, and a piece of it), which moves by the same step each time.  (Slots are
    // below 2^31, and a thread's last places, past them, need the 32nd bit.)
    const int first = part * kThreads + threadIdx.x;
    unsigned slot = first / heads;
    int piece = first % heads;
    while (slot < (unsigned)slots) {
      T x[kAhead];
      int64_t off[kAhead];
      bool live[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        live[k] = slot < (unsigned)slots;
        off[k] = slot * c.slot + (flat ? piece : piece / c.per_head * c.head + piece % c.per_head);
        if (live[k]) x[k] = src[off[k]];
        slot += step_slots;
        piece += step_rest;
        if (piece >= heads) {
          piece -= heads;
          ++slot;
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (live[k]) dst[off[k]] = x[k];
    }
  }
}

// The widest piece that heads, strides and addresses are made of.
template <class Args>
int piece_bytes(const Args& a) {
  const uint64_t bits = (uint64_t)reinterpret_cast<uintptr_t>(a.k_cache) | (uint64_t)reinterpret_cast<uintptr_t>(a.v_cache) |
                        (uint64_t)(2 * a.D) | (uint64_t)(2 * a.layer_stride) | (uint64_t)(2 * a.page_stride) |
                        (uint64_t)(2 * a.slot_stride) | (uint64_t)(2 * a.head_stride);
  return bits & 2 ? 2 : bits & 4 ? 4 : bits & 8 ? 8 : 16;
}

template <class Args>
CacheShape shape_of(const Args& a, int bytes) {
  const int n = bytes / 2;
  return CacheShape{a.layer_stride / n, a.page_stride / n, a.slot_stride / n, a.head_stride / n, a.D / n};
}

// The checks that both calls share.
template <class Args>
int check_cache(const Args& a) {
  if (a.dtype != CLSAMPLE_T_BF16 && a.dtype != CLSAMPLE_T_F16) return CLSAMPLE_ERR_DTYPE;
  if (a.layers < 1 || a.Hkv < 1 || a.D < 1 || a.D > 256 || a.num_pages < 0 || a.page_size < 1 ||
      (int64_t)a.layers * a.Hkv > 0x7fffffff / 512)
    return CLSAMPLE_ERR_SHAPE;
  return CLSAMPLE_SUCCESS;
}

template <int kBytes>
void launch_keep(const clsample_keep_path_args_t& a, cudaStream_t st) {
  const CacheShape c = shape_of(a, kBytes);
  const int64_t columns = (int64_t)2 * a.layers * a.Hkv * c.per_head;
  // two columns a thread: 192 requests' paths in 8 layers (2 x 7.8 MB) 5.5 us, with one 6.6
  int64_t parts = (columns + 2 * kThreads - 1) / (2 * kThreads);
  const int64_t most = (1 << 30) / (int64_t)a.B;
  if (parts > most) parts = most;
  keep_path_kernel<kBytes><<<(unsigned)(a.B * parts), kThreads, 0, st>>>(a, c, (int)parts);
}

// Few copies are shared out among as many CTAs as their pieces take, up to the device's room.
template <int kBytes>
int launch_copy(const clsample_copy_pages_args_t& a, int sms, cudaStream_t st) {
  constexpr int kPerSm = 6;
  const CacheShape c = shape_of(a, kBytes);
  const int64_t pieces = (int64_t)a.page_size * a.Hkv * c.per_head, planes = (int64_t)a.n * 2 * a.layers;
  const int64_t most = (pieces + 8 * kThreads - 1) / (8 * kThreads), room = (int64_t)sms * kPerSm;
  int64_t parts = (room + planes - 1) / planes;
  if (parts > most) parts = most;
  if (parts > 64) parts = 64;
  const int64_t items = planes * parts;
  copy_pages_kernel<kBytes><<<(unsigned)(items < room ? items : room), kThreads, 0, st>>>(a, c, (int)parts);
  return CLSAMPLE_SUCCESS;
}

}  // namespace
}  // namespace clsample

extern "C" {

int clsample_keep_path(const clsample_keep_path_args_t* a, clsample_stream_t stream) {
  using namespace clsample;
  if (!a) return CLSAMPLE_ERR_NULL;
  if (a->B < 0 || a->B > (1 << 24) - 1 || a->N < 0) return CLSAMPLE_ERR_BATCH;
  int rc = check_cache(*a);
  if (rc != CLSAMPLE_SUCCESS) return rc;
  if (a->max_pages < 0 || a->max_path < 0 || a->max_path > kMaxPath) return CLSAMPLE_ERR_SHAPE;
  if (a->table_stride < a->max_pages || a->path_stride < a->max_path) return CLSAMPLE_ERR_STRIDE;
  if (a->B == 0) return CLSAMPLE_SUCCESS;
  if (!a->cu_draft || !a->kv_lens || !a->accepted || !a->new_lens || (!a->page_table && a->max_pages > 0) ||
      (!a->path && a->max_path > 0) || (a->num_pages > 0 && (!a->k_cache || !a->v_cache)))
    return CLSAMPLE_ERR_NULL;
  if (a->new_lens == a->kv_lens) return CLSAMPLE_ERR_SHAPE;
  if ((rc = check_device()) != CLSAMPLE_SUCCESS) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (piece_bytes(*a)) {
    case 16: launch_keep<16>(*a, st); break;
    case 8: launch_keep<8>(*a, st); break;
    case 4: launch_keep<4>(*a, st); break;
    default: launch_keep<2>(*a, st);
  }
  return cudaGetLastError() == cudaSuccess ? CLSAMPLE_SUCCESS : CLSAMPLE_ERR_CUDA;
}

int clsample_copy_pages(const clsample_copy_pages_args_t* a, clsample_stream_t stream) {
  using namespace clsample;
  if (!a) return CLSAMPLE_ERR_NULL;
  if (a->n < 0 || a->n > (1 << 24) - 1) return CLSAMPLE_ERR_BATCH;
  int rc = check_cache(*a);
  if (rc != CLSAMPLE_SUCCESS) return rc;
  if (a->n == 0) return CLSAMPLE_SUCCESS;
  if (!a->copies || (a->num_pages > 0 && (!a->k_cache || !a->v_cache))) return CLSAMPLE_ERR_NULL;
  int sms = 0;
  if ((rc = check_device(nullptr, &sms)) != CLSAMPLE_SUCCESS) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (piece_bytes(*a)) {
    case 16: rc = launch_copy<16>(*a, sms, st); break;
    case 8: rc = launch_copy<8>(*a, sms, st); break;
    case 4: rc = launch_copy<4>(*a, sms, st); break;
    default: rc = launch_copy<2>(*a, sms, st);
  }
  if (rc != CLSAMPLE_SUCCESS) return rc;
  return cudaGetLastError() == cudaSuccess ? CLSAMPLE_SUCCESS : CLSAMPLE_ERR_CUDA;
}

}  // extern "C"
