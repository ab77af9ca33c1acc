// clsample_kv_append: norm of queries and keys per head, position rotation and append of
// keys and values to a paged cache, in one pass (formulas in include/clsample.h).
//
// Bound by memory: (Hq + 2 Hkv) D elements are read once and written once per token, with
// about ten operations each.
#include "paged.cuh"

namespace clsample {
namespace {

constexpr int kThreads = 256;

struct AppendParams {
  clsample_kv_append_args_t a;
};

// The sequence that owns row t, by a 32-way search of the offsets in one warp: the last b
// with cu[b] <= t, if t < cu[b + 1]; -1 when no sequence owns the row.  Offsets out of
// order can only give a wrong or no owner; load_seq and the caller's check t against it.
__device__ __forceinline__ int owner_of(const int32_t* cu, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;  // the owner is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool le = at < hi && __ldg(cu + at) <= t;
    const unsigned m = __ballot_sync(~0u, le);
    if (!(m & 1u)) return -1;
    const int j = 31 - __clz(m);
    lo = lo + j * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

struct Token {
  int b, pos, page, slot;
  bool ok;  // in a sequence, at a position with a cos/sin row and a valid page
};

__device__ __forceinline__ Token find_token(const clsample_kv_append_args_t& a, int t) {
  Token k{-1, 0, 0, 0, false};
  k.b = owner_of(a.cu_new, a.B, t);
  if (k.b < 0) return k;
  const Seq s = load_seq(a.cu_new, a.kv_lens, k.b, a.T, capacity_of(a.max_pages, a.page_size), a.T);
  if (t < s.q0 || t >= s.q0 + s.n) {
    k.b = -1;
    return k;
  }
  if (!s.ok) return k;
  k.pos = s.len - s.n + (t - s.q0);
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
__global__ void __launch_bounds__(kThreads) append_any_kernel(AppendParams P) {
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

// Head rows in 16-byte pieces: lane l of a group of G lanes holds elements 8l .. 8l + 7 of a
// row, so the norm is a reduction over the group and the half-split rotation one exchange
// between lanes.  One block per token: all of a token's rows are in flight at once, and
// while they are, each warp finds the token's sequence, position and page.
template <class T, int G>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendParams P) {
  const clsample_kv_append_args_t& a = P.a;
  constexpr int kGroups = kThreads / G;
  constexpr int kUnroll = 4;
  const int t = blockIdx.x;
  const int group = threadIdx.x / G, l = threadIdx.x % G;
  const bool in = l * 8 < a.D;
  const int heads = a.Hq + 2 * a.Hkv;
  Token k;
  bool found = false;
  for (int r0 = 0; r0 < heads && t < a.T; r0 += kGroups * kUnroll) {
    uint4 raw[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int r = r0 + i * kGroups + group;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (r < heads && in) {
        const T* src = r < a.Hq ? (const T*)a.q + (int64_t)t * a.q_stride_t + (int64_t)r * a.q_stride_h
                       : r < a.Hq + a.Hkv
                           ? (const T*)a.k + (int64_t)t * a.k_stride_t + (int64_t)(r - a.Hq) * a.k_stride_h
                           : (const T*)a.v + (int64_t)t * a.v_stride_t + (int64_t)(r - a.Hq - a.Hkv) * a.v_stride_h;
        raw[i] = *reinterpret_cast<const uint4*>(src + l * 8);
      }
    }
    if (!found) {
      k = find_token(a, t);
      found = true;
    }
    if (k.b < 0) break;
    // the lane's cosines and sines: pairs 8l.. of the half-split form, 4l.. interleaved
    const int half = a.rot_dim / 2;
    const bool turns = k.ok && l * 8 < a.rot_dim;
    float c[8], s[8];
    if (turns) {
      const float* cs = a.cos_sin + (int64_t)k.pos * a.cs_stride;
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c[e] = __ldg(cs + l * 4 + e);
          s[e] = __ldg(cs + half + l * 4 + e);
        }
      } else {
        const int j = l * 8 < half ? l * 8 : l * 8 - half;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          c[e] = __ldg(cs + j + e);
          s[e] = __ldg(cs + half + j + e);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (r0 + i * kGroups >= heads) break;  // uniform over the block
      const int r = r0 + i * kGroups + group;
      const bool is_q = r < a.Hq, is_k = !is_q && r < a.Hq + a.Hkv;
      const int h = is_q ? r : is_k ? r - a.Hq : r - a.Hq - a.Hkv;
      float x[8];
      const uint32_t wds[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = Pair<T>::widen(wds[e]);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
      }
      const T* w = (const T*)(is_q ? a.q_weight : is_k ? a.k_weight : nullptr);
      if (a.q_weight || a.k_weight) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        if (w && in) {
          const float inv = rsqrtf(ss / (float)a.D + a.eps);
          const uint4 wr = __ldg(reinterpret_cast<const uint4*>(w + l * 8));
          const uint32_t ww[4] = {wr.x, wr.y, wr.z, wr.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = Pair<T>::widen(ww[e]);
            x[2 * e] = x[2 * e] * inv * f.x;
            x[2 * e + 1] = x[2 * e + 1] * inv * f.y;
          }
        }
      }
      if (a.rot_dim > 0) {
        if (a.interleaved) {
          if (turns) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = x[2 * e], q = x[2 * e + 1];
              x[2 * e] = p * c[e] - q * s[e];
              x[2 * e + 1] = q * c[e] + p * s[e];
            }
          }
        } else {
          const bool second = l * 8 >= half;
          const int lane = threadIdx.x & 31;
          const int from = l * 8 < a.rot_dim ? (second ? lane - half / 8 : lane + half / 8) : lane;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float o = __shfl_sync(~0u, x[e], from);
            if (turns) x[e] = second ? x[e] * c[e] + o * s[e] : x[e] * c[e] - o * s[e];
          }
        }
      }
      if (r < heads && in) {
        uint4 y = raw[i];
        if (is_q || is_k)
          y = make_uint4(Pair<T>::narrow(x[0], x[1]), Pair<T>::narrow(x[2], x[3]), Pair<T>::narrow(x[4], x[5]),
                         Pair<T>::narrow(x[6], x[7]));
        if (is_q) {
          if (!k.ok) y = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>((T*)a.q_out + (int64_t)t * a.qo_stride_t + (int64_t)h * a.qo_stride_h + l * 8) = y;
        } else if (k.ok) {
          T* cache = (T*)(is_k ? a.k_cache : a.v_cache);
          *reinterpret_cast<uint4*>(cache + (int64_t)k.page * a.page_stride + (int64_t)k.slot * a.slot_stride +
                                    (int64_t)h * a.head_stride + l * 8) = y;
        }
      }
    }
  }
  if (a.row_status)
    for (int b = blockIdx.x * kThreads + threadIdx.x; b < a.B; b += gridDim.x * kThreads) write_status(a, b);
}

template <class T>
void launch_append(const AppendParams& P, bool fast, cudaStream_t st) {
  // without tokens the blocks only write statuses
  const unsigned grid = P.a.T > 0 ? (unsigned)P.a.T : (unsigned)((P.a.B + kThreads - 1) / kThreads);
  if (!fast)
    append_any_kernel<T><<<grid, kThreads, 0, st>>>(P);
  else if (P.a.D <= 64)
    append_kernel<T, 8><<<grid, kThreads, 0, st>>>(P);
  else if (P.a.D <= 128)
    append_kernel<T, 16><<<grid, kThreads, 0, st>>>(P);
  else
    append_kernel<T, 32><<<grid, kThreads, 0, st>>>(P);
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
  const int rc = check_device();
  if (rc != CLSAMPLE_SUCCESS) return rc;
  const int64_t strides = a->q_stride_t | a->q_stride_h | a->k_stride_t | a->k_stride_h | a->v_stride_t |
                          a->v_stride_h | a->qo_stride_t | a->qo_stride_h | a->page_stride | a->slot_stride |
                          a->head_stride;
  const bool fast = a->D % 8 == 0 && a->rot_dim % (a->interleaved ? 8 : 16) == 0 && (strides & 7) == 0 &&
                    aligned16(a->q) && aligned16(a->k) && aligned16(a->v) && aligned16(a->q_out) &&
                    aligned16(a->k_cache) && aligned16(a->v_cache) && aligned16(a->q_weight) && aligned16(a->k_weight);
  const AppendParams P{*a};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a->dtype == CLSAMPLE_T_BF16)
    launch_append<__nv_bfloat16>(P, fast, st);
  else
    launch_append<__half>(P, fast, st);
  return cudaGetLastError() == cudaSuccess ? CLSAMPLE_SUCCESS : CLSAMPLE_ERR_CUDA;
}
