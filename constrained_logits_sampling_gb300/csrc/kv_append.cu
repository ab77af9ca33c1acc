// clsample_kv_append: norm of queries and keys per head, position rotation and append of
// keys and values to a paged cache, in one pass (formulas in include/clsample.h).
//
// Bound by memory: (Hq + 2 Hkv) D elements are read once and written once per token, with
// about ten operations each.  8192 tokens of 32 + 8 heads of 128 bf16 elements (206 MB): 39 us,
// 5.2 TB/s; 1024 tokens with norm (26 MB): 10.3 us; one token: 6.3 to 6.9 us, all of it latency.
#include "paged.cuh"

namespace clsample {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 4;  // of the fast path

constexpr int kMaxTokens = 16;   // of a block
constexpr int kMaxHeads = 256;   // Hq + 2 Hkv of the fast path

struct AppendParams {
  clsample_kv_append_args_t a;
  int tokens;  // of a block of the fast path
};

struct Token {
  int b, pos, page, slot;
  bool ok;  // in a sequence, at a position with a cos/sin row and a valid page
};

// The sequence that owns row t (the last b with cu[b] <= t, if t < cu[b + 1]), the row's
// position, page and slot, by one warp: a 32-way search of the offsets, whose last step reads
// the lengths along.  b is -1 when no sequence owns the row.  Offsets out of order can only
// give a wrong owner or none: what is found is checked against them.
__device__ __forceinline__ Token find_token(const clsample_kv_append_args_t& a, int t) {
  const int lane = threadIdx.x & 31;
  Token k{-1, 0, 0, 0, false};
  int lo = 0, hi = a.B;  // the owner is in [lo, hi)
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const unsigned m = __ballot_sync(~0u, at < hi && __ldg(a.cu_new + at) <= t);
    if (!(m & 1u)) return k;
    lo += (31 - __clz(m)) * step;
    hi = min(hi, lo + step);
  }
  const int at = lo + lane;
  int from = 0, to = 0, len = 0;
  if (at < hi) {
    from = __ldg(a.cu_new + at);
    to = __ldg(a.cu_new + at + 1);
    len = __ldg(a.kv_lens + at);
  }
  const unsigned m = __ballot_sync(~0u, at < hi && from <= t);
  if (!m) return k;
  const int src = 31 - __clz(m);
  from = __shfl_sync(~0u, from, src);
  to = __shfl_sync(~0u, to, src);
  len = __shfl_sync(~0u, len, src);
  if (from < 0 || to > a.T || t < from || t >= to) return k;
  k.b = lo + src;
  if (len < 0 || len > capacity_of(a.max_pages, a.page_size)) return k;
  k.pos = len - (to - from) + (t - from);
  if (k.pos < 0 || (a.rot_dim > 0 && k.pos >= a.max_pos)) return k;
  k.page = __ldg(a.page_table + (int64_t)k.b * a.table_stride + k.pos / a.page_size);
  k.slot = k.pos % a.page_size;
  k.ok = k.page >= 0 && k.page < a.num_pages;
  return k;
}

// Statuses, one thread per sequence: the same checks as find_token for each of its tokens'
// pages.  Runs in the first blocks of the launch, after their token.
__device__ __forceinline__ void write_status(const clsample_kv_append_args_t& a, int b) {
  const int cap = capacity_of(a.max_pages, a.page_size);
  const Seq s = load_seq(a.cu_new, a.kv_lens, b, a.T, cap, a.T);
  bool ok = s.ok;
  if (ok && s.n > 0) {
    const int first = s.len - s.n;
    if (first < 0 || (a.rot_dim > 0 && s.len > a.max_pos)) {
      ok = false;
    } else {
      for (int p = first / a.page_size; ok && p <= (s.len - 1) / a.page_size; ++p) {
        const int id = __ldg(a.page_table + (int64_t)b * a.table_stride + p);
        ok = id >= 0 && id < a.num_pages;
      }
    }
  }
  a.row_status[b] = ok ? CLSAMPLE_ROW_OK : CLSAMPLE_ROW_INVALID;
}

// Any head size, strides and rotation: one warp per head row, elements one by one through
// shared memory.
template <class T>
__global__ void __launch_bounds__(kThreads) append_any_kernel(const __grid_constant__ AppendParams P) {
  const clsample_kv_append_args_t& a = P.a;
  __shared__ float rows[kThreads / 32][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, D = a.D;
  float* x = rows[warp];
  const int heads = a.Hq + 2 * a.Hkv;
  if ((int)blockIdx.x < a.T) {
    const int t = blockIdx.x;
    const Token k = find_token(a, t);
    for (int r = warp; r < heads && k.b >= 0; r += kThreads / 32) {
      const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.Hkv;
      const int h = is_q ? r : is_v ? r - a.Hq - a.Hkv : r - a.Hq;
      T* dst = is_q ? (T*)a.q_out + (int64_t)t * a.qo_stride_t + (int64_t)h * a.qo_stride_h
                    : (T*)(is_v ? a.v_cache : a.k_cache) + (int64_t)k.page * a.page_stride +
                          (int64_t)k.slot * a.slot_stride + (int64_t)h * a.head_stride;
      if (!k.ok) {
        if (is_q)
          for (int d = lane; d < D; d += 32) dst[d] = from_f32<T>(0.f);
        continue;
      }
      const T* src = is_q   ? (const T*)a.q + (int64_t)t * a.q_stride_t + (int64_t)h * a.q_stride_h
                     : is_v ? (const T*)a.v + (int64_t)t * a.v_stride_t + (int64_t)h * a.v_stride_h
                            : (const T*)a.k + (int64_t)t * a.k_stride_t + (int64_t)h * a.k_stride_h;
      if (is_v) {
        for (int d = lane; d < D; d += 32) dst[d] = src[d];
        continue;
      }
      const T* w = (const T*)(is_q ? a.q_weight : a.k_weight);
      float ss = 0.f;
      for (int d = lane; d < D; d += 32) {
        const float e = to_f32(src[d]);
        x[d] = e;
        ss = fmaf(e, e, ss);
      }
      if (w) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        const float inv = rsqrtf(ss / (float)D + a.eps);
        for (int d = lane; d < D; d += 32) x[d] = x[d] * inv * to_f32(w[d]);
      }
      __syncwarp();
      const int half = a.rot_dim / 2;
      const float* cs = a.cos_sin + (int64_t)k.pos * a.cs_stride;
      for (int d = lane; d < D; d += 32) {
        float y = x[d];
        if (d < a.rot_dim) {
          const int j = a.interleaved ? d >> 1 : d < half ? d : d - half;
          const bool second = a.interleaved ? d & 1 : d >= half;
          const float c = __ldg(cs + j), s = __ldg(cs + half + j);
          const float o = a.interleaved ? x[d ^ 1] : x[second ? d - half : d + half];
          y = second ? y * c + o * s : y * c - o * s;
        }
        dst[d] = from_f32<T>(y);
      }
      __syncwarp();
    }
  }
  if (a.row_status)
    for (int b = blockIdx.x * kThreads + threadIdx.x; b < a.B; b += gridDim.x * kThreads) write_status(a, b);
}

// Where a head row comes from and goes to, for the block's first token.
struct HeadRow {
  const unsigned char* src;
  unsigned char* dst;  // of k and v: of the cache's first slot
  int64_t src_stride;  // bytes from a token to the next
  int kind;            // 0 q, 1 k, 2 v
};

// Head rows in 16-byte pieces: lane l of a group of G lanes holds elements 8l .. 8l + 7 of a
// row, so the norm is a reduction over the group and the half-split rotation one exchange
// between lanes.  A block takes a few consecutive tokens.  Its first head rows are on their way
// while the warps find its tokens' sequences, positions and pages; from then on a token's rows
// are loaded while the one before it is worked on.  Addresses come from a table in shared
// memory: with the selection between q, k and v in each row the instructions took longer than
// the memory (8192 tokens, on an earlier version: 68 us, 52 with the table).
// kPaired, for the usual case of a whole head rotated in halves: lane l has elements 4l .. 4l + 3
// of both halves instead, so that pairs meet in a lane and nothing is exchanged (8192
// tokens: 38 us against 43; 1024 with norm: 10.4 against 12.3).
template <class T, int G, bool kPaired>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) append_kernel(const __grid_constant__ AppendParams P) {
  const clsample_kv_append_args_t& a = P.a;
  constexpr int kGroups = kThreads / G;
  constexpr int kUnroll = 3;  // head rows of a group in flight
  __shared__ Token tokens[kMaxTokens];
  __shared__ HeadRow table[kMaxHeads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = tid / G, l = tid % G;
  const bool in = l * 8 < a.D;
  const int heads = a.Hq + 2 * a.Hkv;
  const int t0 = blockIdx.x * P.tokens, count = min(P.tokens, a.T - t0);
  const int half = a.rot_dim / 2;

  for (int r = tid; r < heads; r += kThreads) {
    const int kind = r < a.Hq ? 0 : r < a.Hq + a.Hkv ? 1 : 2;
    const int h = kind == 0 ? r : kind == 1 ? r - a.Hq : r - a.Hq - a.Hkv;
    const T* src = (const T*)(kind == 0 ? a.q : kind == 1 ? a.k : a.v);
    const int64_t st = kind == 0 ? a.q_stride_t : kind == 1 ? a.k_stride_t : a.v_stride_t;
    const int64_t hd = kind == 0 ? a.q_stride_h : kind == 1 ? a.k_stride_h : a.v_stride_h;
    T* dst = (T*)(kind == 0 ? a.q_out : kind == 1 ? a.k_cache : a.v_cache);
    table[r] = HeadRow{(const unsigned char*)(src + t0 * st + h * hd),
                       (unsigned char*)(kind == 0 ? dst + t0 * a.qo_stride_t + h * a.qo_stride_h : dst + h * a.head_stride),
                       st * (int64_t)sizeof(T), kind};
  }
  __syncthreads();

  uint4 raw[kUnroll];
  auto fetch = [&](int token, int r0) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int r = r0 + i * kGroups + group;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (r < heads && in) {
        const unsigned char* src = table[r].src + token * table[r].src_stride;
        if (kPaired) {
          const uint2 x = *reinterpret_cast<const uint2*>(src + l * 8);
          const uint2 y = *reinterpret_cast<const uint2*>(src + a.D + l * 8);  // D / 2 elements further
          raw[i] = make_uint4(x.x, x.y, y.x, y.y);
        } else {
          raw[i] = *reinterpret_cast<const uint4*>(src + l * 16);
        }
      }
    }
  };
  if (count > 0) fetch(0, 0);
  for (int i = warp; i < count; i += kThreads / 32) {
    const Token k = find_token(a, t0 + i);
    if (lane == 0) tokens[i] = k;
  }
  __syncthreads();

  // the lane that holds the other elements of this one's pairs; where it is the second of them
  const bool second = !a.interleaved && l * 8 >= half;
  const int from = !a.interleaved && l * 8 < a.rot_dim ? (second ? lane - half / 8 : lane + half / 8) : lane;
  const int turn_at = kPaired || a.interleaved ? l * 4 : second ? l * 8 - half : l * 8;
  const bool norm = a.q_weight || a.k_weight;

  for (int token = 0, r0 = 0; token < count;) {
    const Token& k = tokens[token];
    uint4 now[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) now[i] = raw[i];
    const int this_r0 = r0, this_token = token;
    r0 += kGroups * kUnroll;
    if (r0 >= heads) {
      r0 = 0;
      ++token;
    }
    if (token < count) fetch(token, r0);
    if (k.b < 0) continue;
    const bool turns = k.ok && l * 8 < a.rot_dim;
    float c[8], s[8];  // cosines; sines, negative for the first elements of pairs
    if (turns) {
      const float* cs = a.cos_sin + (int64_t)k.pos * a.cs_stride + turn_at;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (e == 0 || (!kPaired && !a.interleaved)) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(cs + 4 * e));
          const float4 y = __ldg(reinterpret_cast<const float4*>(cs + half + 4 * e));
          const float sign = kPaired || second || a.interleaved ? 1.f : -1.f;
          c[4 * e] = x.x, c[4 * e + 1] = x.y, c[4 * e + 2] = x.z, c[4 * e + 3] = x.w;
          s[4 * e] = y.x * sign, s[4 * e + 1] = y.y * sign, s[4 * e + 2] = y.z * sign, s[4 * e + 3] = y.w * sign;
        }
      }
    }
    const int64_t cache_at = ((int64_t)k.page * a.page_stride + (int64_t)k.slot * a.slot_stride) * (int64_t)sizeof(T);
    const int64_t out_at = this_token * a.qo_stride_t * (int64_t)sizeof(T);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int r = this_r0 + i * kGroups + group;
      if (r - group >= heads) break;  // uniform over the block
      const int kind = r < heads ? table[r].kind : 2;
      uint4 y = now[i];
      if (__any_sync(~0u, kind < 2)) {  // not a warp of values
        float x[8];
        const uint32_t wds[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = Pair<T>::widen(wds[e]);
          x[2 * e] = f.x;
          x[2 * e + 1] = f.y;
        }
        if (norm) {
          const T* w = (const T*)(kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr);
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
          for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
          if (w && in) {
            const float inv = rsqrtf(ss / (float)a.D + a.eps);
            const uint2 wa = __ldg(reinterpret_cast<const uint2*>(kPaired ? w + l * 4 : w + l * 8));
            const uint2 wb = __ldg(reinterpret_cast<const uint2*>(kPaired ? w + half + l * 4 : w + l * 8 + 4));
            const uint32_t ww[4] = {wa.x, wa.y, wb.x, wb.y};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = Pair<T>::widen(ww[e]);
              x[2 * e] = x[2 * e] * inv * f.x;
              x[2 * e + 1] = x[2 * e + 1] * inv * f.y;
            }
          }
        }
        if (kPaired) {
          if (turns) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = x[e], q = x[e + 4];
              x[e] = p * c[e] - q * s[e];
              x[e + 4] = q * c[e] + p * s[e];
            }
          }
        } else if (a.interleaved) {
          if (turns) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = x[2 * e], q = x[2 * e + 1];
              x[2 * e] = p * c[e] - q * s[e];
              x[2 * e + 1] = q * c[e] + p * s[e];
            }
          }
        } else if (half > 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float o = __shfl_sync(~0u, x[e], from);
            if (turns) x[e] = x[e] * c[e] + o * s[e];
          }
        }
        if (kind < 2)
          y = make_uint4(Pair<T>::narrow(x[0], x[1]), Pair<T>::narrow(x[2], x[3]), Pair<T>::narrow(x[4], x[5]),
                         Pair<T>::narrow(x[6], x[7]));
      }
      if (r < heads && in && (k.ok || kind == 0)) {
        if (!k.ok) y = make_uint4(0, 0, 0, 0);
        unsigned char* dst = table[r].dst + (kind == 0 ? out_at : cache_at);
        if (kPaired) {
          *reinterpret_cast<uint2*>(dst + l * 8) = make_uint2(y.x, y.y);
          *reinterpret_cast<uint2*>(dst + a.D + l * 8) = make_uint2(y.z, y.w);
        } else {
          *reinterpret_cast<uint4*>(dst + l * 16) = y;
        }
      }
    }
  }
  if (a.row_status)
    for (int b = blockIdx.x * kThreads + tid; b < a.B; b += gridDim.x * kThreads) write_status(a, b);
}

template <class T>
void launch_append(AppendParams P, bool fast, int sms, cudaStream_t st) {
  // without tokens the blocks only write statuses
  const int status_blocks = (P.a.B + kThreads - 1) / kThreads;
  if (!fast) {
    append_any_kernel<T><<<P.a.T > 0 ? P.a.T : status_blocks, kThreads, 0, st>>>(P);
    return;
  }
  // as many tokens a block as it takes for the blocks to fit the device at once (8192 tokens: 38 us,
  // with one token a block 50)
  P.tokens = (P.a.T + sms * kBlocksPerSm - 1) / (sms * kBlocksPerSm);
  P.tokens = P.tokens < 1 ? 1 : P.tokens > kMaxTokens ? kMaxTokens : P.tokens;
  const int grid = P.a.T > 0 ? (P.a.T + P.tokens - 1) / P.tokens : status_blocks;
  const bool paired = P.a.rot_dim == P.a.D && !P.a.interleaved;
  auto* fn = P.a.D <= 64    ? (paired ? append_kernel<T, 8, true> : append_kernel<T, 8, false>)
             : P.a.D <= 128 ? (paired ? append_kernel<T, 16, true> : append_kernel<T, 16, false>)
                            : (paired ? append_kernel<T, 32, true> : append_kernel<T, 32, false>);
  fn<<<grid, kThreads, 0, st>>>(P);
}

}  // namespace
}  // namespace clsample

extern "C" int clsample_kv_append(const clsample_kv_append_args_t* a, clsample_stream_t stream) {
  using namespace clsample;
  if (!a) return CLSAMPLE_ERR_NULL;
  if (a->B < 0 || a->B > (1 << 24) - 1 || a->T < 0 || a->T > kMaxLen) return CLSAMPLE_ERR_BATCH;
  if (a->dtype != CLSAMPLE_T_BF16 && a->dtype != CLSAMPLE_T_F16) return CLSAMPLE_ERR_DTYPE;
  if (a->Hq < 0 || a->Hkv < 1 || a->Hq > 65536 || a->Hkv > 65536 || a->D < 1 || a->D > 256 || a->num_pages < 0 ||
      a->page_size < 1 || a->max_pages < 0 || a->rot_dim < 0 || a->rot_dim > a->D || (a->rot_dim & 1) ||
      a->max_pos < 0 || !(a->eps >= 0.f))
    return CLSAMPLE_ERR_SHAPE;
  if (a->table_stride < a->max_pages || (a->rot_dim > 0 && a->cs_stride < a->rot_dim)) return CLSAMPLE_ERR_STRIDE;
  if (a->B == 0 || (a->T == 0 && !a->row_status)) return CLSAMPLE_SUCCESS;
  if (!a->cu_new || !a->kv_lens || (!a->page_table && a->max_pages > 0)) return CLSAMPLE_ERR_NULL;
  if (a->T > 0 && (!a->k || !a->v || !a->k_cache || !a->v_cache || (a->Hq > 0 && (!a->q || !a->q_out)) ||
                   (a->rot_dim > 0 && !a->cos_sin)))
    return CLSAMPLE_ERR_NULL;
  int sms = 0;
  const int rc = check_device(nullptr, &sms);
  if (rc != CLSAMPLE_SUCCESS) return rc;
  const int64_t strides = a->q_stride_t | a->q_stride_h | a->k_stride_t | a->k_stride_h | a->v_stride_t |
                          a->v_stride_h | a->qo_stride_t | a->qo_stride_h | a->page_stride | a->slot_stride |
                          a->head_stride;
  const bool fast = a->Hq + 2 * a->Hkv <= kMaxHeads && a->D % 8 == 0 && a->rot_dim % (a->interleaved ? 8 : 16) == 0 && (strides & 7) == 0 &&
                    aligned16(a->q) && aligned16(a->k) && aligned16(a->v) && aligned16(a->q_out) &&
                    aligned16(a->k_cache) && aligned16(a->v_cache) && aligned16(a->q_weight) && aligned16(a->k_weight) &&
                    aligned16(a->cos_sin) && a->cs_stride % 4 == 0;
  const AppendParams P{*a, 1};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a->dtype == CLSAMPLE_T_BF16)
    launch_append<__nv_bfloat16>(P, fast, sms, st);
  else
    launch_append<__half>(P, fast, sms, st);
  return cudaGetLastError() == cudaSuccess ? CLSAMPLE_SUCCESS : CLSAMPLE_ERR_CUDA;
}
