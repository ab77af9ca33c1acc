// Attention for few query rows per key head: bound by reading keys and values once.
//
// A unit is 16 packed rows (attn_units.cuh).  Four warps share the rows and split the keys: of
// each tile of 64 keys a warp takes 16, loads them itself (cp.async, its own ring of stages) and
// keeps its own running maximum, sum and output in registers, so no barrier stands between a
// load and its use and every byte passes shared memory once.  The products are mma.m16n8k16:
// with so few rows the tensor cores are nearly idle either way, and the row tile can be 16 where
// tcgen05 has 64 at least.  The four warps' results meet in shared memory at the end of a
// unit's span.  256 requests of 4 tokens on 32 / 8 heads of 128 over 200 to 4000 keys (2.27 GB):
// 386 us, 5.9 TB/s, with rows of 256 bytes 2 KB apart in the cache; one token over 777 keys: 12 us.
// A warp of its own that copied by TMA, on into the next unit while the others ended one, was no
// faster (on an earlier version, 407 us against 404) and slower where a unit is one tile (19 and 15).
#pragma once

#include "attn_units.cuh"

namespace clsample {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
// An arrival on `bar` once all of this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <class T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr int kStreamThreads = 128;
constexpr int kStreamKeys = 64;
constexpr float kLn2 = 0.693147180559945309f;

// Ring stages of a warp: two CTAs fit an SM, with up to 128 KB of loads in flight for heads of 128
// and 160 KB for heads of 64 (all stages but the one that is worked on).
constexpr int kStreamRows = 16;
template <int D>
struct StreamRing {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kBytes = kStages * kStreamKeys * D * 2 * 2;  // keys and values
  static_assert(kBytes >= 4 * kStreamRows * (D + 8) * 4, "room for four warps' sums");
};

// A scratch slot: R x D sums, then R maxima (log2 units) and R weights' sums.
template <int R, int D>
__device__ __forceinline__ float* scratch_slot(const AttnParams& P, int cta, int which) {
  return P.partial + (int64_t)(cta * 2 + which) * (R * (D + 2));
}

// Writes four output elements of a packed row.
template <class T>
__device__ __forceinline__ void store_out4(const AttnParams& P, const Unit& u, int r, int d, float4 o) {
  const int row = u.row0 + r;
  T* dst = (T*)P.a.out + (int64_t)(u.q0 + token_of(P, row)) * P.a.o_stride_t +
           (int64_t)(u.h * P.g + head_of(P, row)) * P.a.o_stride_h + d;
  *reinterpret_cast<uint2*>(dst) = make_uint2(Pair<T>::narrow(o.x, o.y), Pair<T>::narrow(o.z, o.w));
}
__device__ __forceinline__ float lse_of(float m, float l) {  // m in log2 units
  return l > 0.f || l != l ? (m + log2f(l)) * kLn2 : __int_as_float(0xff800000);
}
__device__ __forceinline__ void store_lse(const AttnParams& P, const Unit& u, int r, float m, float l) {
  const int row = u.row0 + r;
  if (P.a.lse) P.a.lse[(int64_t)(u.q0 + token_of(P, row)) * P.a.Hq + u.h * P.g + head_of(P, row)] = lse_of(m, l);
}

// The rows of a unit as one warp has them: queries as A operands, limits and running sums.  Lane
// i has rows i / 4 and i / 4 + 8.
template <class T, int D>
struct StreamState {
  uint32_t q[D / 16][4];
  int pos[2];
  int pos_first, pos_last;
  float o[D / 8][4];
  float m[2], l[2];

  __device__ __forceinline__ void begin(const AttnParams& P, const Unit& u) {
    const int lane = threadIdx.x & 31;
    const float neg_inf = __int_as_float(0xff800000);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = hf * 8 + (lane >> 2);
      const bool live = r < u.rows;
      const int row = u.row0 + r;
      const T* src = (const T*)P.a.q + (int64_t)(u.q0 + (live ? token_of(P, row) : 0)) * P.a.q_stride_t +
                     (int64_t)(u.h * P.g + (live ? head_of(P, row) : 0)) * P.a.q_stride_h + (lane & 3) * 2;
      pos[hf] = live ? u.len - u.n + token_of(P, row) : -1;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        q[ks][hf] = live ? __ldg(reinterpret_cast<const unsigned*>(src + ks * 16)) : 0u;
        q[ks][hf + 2] = live ? __ldg(reinterpret_cast<const unsigned*>(src + ks * 16 + 8)) : 0u;
      }
      m[hf] = neg_inf;
      l[hf] = 0.f;
    }
    pos_first = u.len - u.n + token_of(P, u.row0);
    pos_last = u.len - u.n + token_of(P, u.row0 + u.rows - 1);
#pragma unroll
    for (int d = 0; d < D / 8; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
  }

  // 16 keys from position `key` on, of which those in `live` exist.  Rows of 64 elements in
  // shared memory, 16-byte pieces swizzled by the row; the next 64 elements are `half` further.
  __device__ __forceinline__ void step(const AttnParams& P, uint32_t kb, uint32_t vb, uint32_t half, int key,
                                       unsigned live) {
    const int lane = threadIdx.x & 31;
    const float neg_inf = __int_as_float(0xff800000);
    float s[2][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[0][e] = s[1][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const int row = (lane & 7) + ((lane >> 4) << 3), ch = ks * 2 + ((lane >> 3) & 1);
      uint32_t b[4];
      ldmatrix4(b, kb + (ch >> 3) * half + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
      mma16816<T>(s[0], q[ks], b[0], b[1]);
      mma16816<T>(s[1], q[ks], b[2], b[3]);
    }
    const int window = P.a.window;
    // every key of the tile is seen by every row (rows past the unit's are never stored)
    const bool whole = live == 0xffffu && key + 15 <= pos_first && (window <= 0 || key > pos_last - window);
    bool moved = false;
    float keep[2];
    uint32_t p[4];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float x[4] = {s[0][hf * 2] * P.scale_log2, s[0][hf * 2 + 1] * P.scale_log2, s[1][hf * 2] * P.scale_log2,
                    s[1][hf * 2 + 1] * P.scale_log2};
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = (e >> 1) * 8 + (lane & 3) * 2 + (e & 1);
          const int kp = key + c;
          if (!((live >> c) & 1) || kp > pos[hf] || (window > 0 && kp <= pos[hf] - window)) x[e] = neg_inf;
        }
      }
      float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      const float mn = fmaxf(m[hf], top);
      const float base = mn == neg_inf ? 0.f : mn;  // a row that has seen no key yet
      keep[hf] = exp2_fast(m[hf] - base);
      moved |= mn != m[hf];
      m[hf] = mn;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = exp2_fast(x[e] - base);
        sum += x[e];
      }
      l[hf] = l[hf] * keep[hf] + sum;
      p[hf] = Pair<T>::narrow(x[0], x[1]);
      p[hf + 2] = Pair<T>::narrow(x[2], x[3]);
    }
    if (__any_sync(~0u, moved)) {
#pragma unroll
      for (int d = 0; d < D / 8; ++d) {
        o[d][0] *= keep[0];
        o[d][1] *= keep[0];
        o[d][2] *= keep[1];
        o[d][3] *= keep[1];
      }
    }
    // values of keys that do not exist may be anything, and 0 x NaN is NaN
    const unsigned two = live >> ((lane & 3) * 2);
    const uint32_t mask0 = (two & 1 ? 0xffffu : 0u) | (two & 2 ? 0xffff0000u : 0u);
    const uint32_t mask1 = (two & 0x100 ? 0xffffu : 0u) | (two & 0x200 ? 0xffff0000u : 0u);
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      const int row = (lane & 7) + (((lane >> 3) & 1) << 3), ch = d * 2 + (lane >> 4);
      uint32_t b[4];
      ldmatrix4_trans(b, vb + (ch >> 3) * half + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
      mma16816<T>(o[2 * d], p, b[0] & mask0, b[1] & mask1);
      mma16816<T>(o[2 * d + 1], p, b[2] & mask0, b[3] & mask1);
    }
  }
};

// The warps' results of a unit's span meet: meet holds [warp][row][D + 8] (rows begin in different
// banks), wm and wl the warps' maxima and sums.
template <class T, int D>
__device__ __forceinline__ void stream_finish(const AttnParams& P, const Unit& u, StreamState<T, D>& st, float* meet,
                                              float (&wm)[4][kStreamRows], float (&wl)[4][kStreamRows], bool done,
                                              float* slot) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int R = kStreamRows;
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    float sum = st.l[hf];
    sum += __shfl_xor_sync(~0u, sum, 1);
    sum += __shfl_xor_sync(~0u, sum, 2);
    if ((lane & 3) == 0) {
      wm[warp][hf * 8 + (lane >> 2)] = st.m[hf];
      wl[warp][hf * 8 + (lane >> 2)] = sum;
    }
  }
#pragma unroll
  for (int d = 0; d < D / 8; ++d)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int col = d * 8 + (lane & 3) * 2, row = hf * 8 + (lane >> 2);
      *reinterpret_cast<float2*>(meet + (warp * R + row) * (D + 8) + col) =
          make_float2(st.o[d][hf * 2], st.o[d][hf * 2 + 1]);
    }
  __syncthreads();
  for (int i = tid; i < u.rows * (D / 4); i += kStreamThreads) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    const float top = fmaxf(fmaxf(wm[0][r], wm[1][r]), fmaxf(wm[2][r], wm[3][r]));
    const float base = top == __int_as_float(0xff800000) ? 0.f : top;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float lsum = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = exp2_fast(wm[w][r] - base);
      const float4 v = *reinterpret_cast<const float4*>(meet + (w * R + r) * (D + 8) + d);
      sum = make_float4(sum.x + v.x * f, sum.y + v.y * f, sum.z + v.z * f, sum.w + v.w * f);
      lsum += wl[w][r] * f;
    }
    if (done) {
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
      store_out4<T>(P, u, r, d, make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
      if (d == 0) store_lse(P, u, r, top, lsum);
    } else {
      __stcg(reinterpret_cast<float4*>(slot + r * D + d), sum);
      if (d == 0) {
        __stcg(slot + R * D + r, top);
        __stcg(slot + R * D + R + r, lsum);
      }
    }
  }
  __syncthreads();  // for the next unit
}

template <class T, int D>
__global__ void __launch_bounds__(kStreamThreads, 2) attn_stream_kernel(const __grid_constant__ AttnParams P) {
  constexpr int R = kStreamRows, S = StreamRing<D>::kStages, KC = D / 8;  // KC: 16-byte pieces of a key
  constexpr int kTileBytes = 16 * D * 2, kStageBytes = 2 * kTileBytes, kHalf = 16 * 128;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ unsigned key_ok[4][S];
  __shared__ float wm[4][R], wl[4][R];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const clsample_attention_args_t& a = P.a;
  const uint32_t ring_addr = static_cast<uint32_t>(__cvta_generic_to_shared(smem + warp * S * kStageBytes));

  let_next_grid_start();
  Span span;
  Unit u;
  int64_t unit_begin;
  if (!find_span<R, kStreamKeys, kStreamThreads>(P, &span, &u, &unit_begin)) {
    if (tid == 0) P.cut[blockIdx.x].rows = 0;
    wait_for_earlier_grids();  // this grid's end stands for theirs
    return;
  }

  int64_t t = span.t0;
  while (true) {
    const int j0 = (int)(t - unit_begin);
    const int cnt = (int)min((int64_t)(u.tiles - j0), span.t1 - t);
    if (tid == 0 && t + cnt >= span.t1) note_cut(P, span, u, unit_begin);
    const T* kc = (const T*)a.k_cache + (int64_t)u.h * a.head_stride;
    const T* vc = (const T*)a.v_cache + (int64_t)u.h * a.head_stride;
    const int32_t* table = a.page_table + (int64_t)u.b * a.table_stride;
    const int key0 = (u.tile0 + j0) * kStreamKeys + warp * 16;  // the warp's first key

    // the page of this lane's key (lanes 0..15) in the span's tile i; -1: not to be read
    auto page_of = [&](int i) {
      const int key = key0 + i * kStreamKeys + (lane & 15);
      if (i >= cnt || key < u.key_lo || key >= u.key_hi) return -1;
      const int id = __ldg(table + (P.page_shift >= 0 ? key >> P.page_shift : key / a.page_size));
      return id < a.num_pages ? id : -1;
    };
    auto issue = [&](int i, int page) {
      const int stage = i % S;
      const int key = key0 + i * kStreamKeys + (lane & 15);
      const int slot = P.page_shift >= 0 ? key & ((1 << P.page_shift) - 1) : key % a.page_size;
      const bool ok = page >= 0;
      const int64_t off = ok ? (int64_t)page * a.page_stride + (int64_t)slot * a.slot_stride : 0;
      const unsigned mask = __ballot_sync(~0u, ok) & 0xffffu;
      if (lane == 0) key_ok[warp][stage] = mask;
      const uint32_t base = ring_addr + stage * kStageBytes;
      if (i < cnt) {
#pragma unroll
        for (int x = 0; x < KC / 2; ++x) {
          const int row = (x * 32 + lane) / KC, ch = (x * 32 + lane) % KC;
          const int64_t o = __shfl_sync(~0u, off, row) + ch * 8;
          const bool live = (mask >> row) & 1;
          const uint32_t dst = base + (ch >> 3) * kHalf + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
          cp_async16(dst, kc + o, live);
          cp_async16(dst + kTileBytes, vc + o, live);
        }
      }
      cp_async_commit();
    };

    // the first stages are on their way before the queries are read
    int page = page_of(0);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      const int next = page_of(i + 1);
      issue(i, page);
      page = next;
    }
    StreamState<T, D> st;
    st.begin(P, u);
    for (int i = 0; i < cnt; ++i) {
      cp_async_wait<S - 2>();
      __syncwarp();
      const int next = page_of(i + S);
      issue(i + S - 1, page);
      page = next;
      const int stage = i % S;
      const uint32_t kb = ring_addr + stage * kStageBytes;
      st.step(P, kb, kb + kTileBytes, kHalf, key0 + i * kStreamKeys, key_ok[warp][stage]);
    }
    cp_async_wait<0>();
    __syncthreads();  // the rings are drained: the first is where the warps meet
    stream_finish<T, D>(P, u, st, reinterpret_cast<float*>(smem), wm, wl, cnt == u.tiles,
                                   scratch_slot<R, D>(P, blockIdx.x, j0 == 0 ? 1 : 0));
    t += cnt;
    if (t >= span.t1) break;
    unit_begin = t;
    next_unit<R, kStreamKeys>(P, &u);
  }
  wait_for_earlier_grids();  // this grid's end stands for theirs
}

}  // namespace clsample
