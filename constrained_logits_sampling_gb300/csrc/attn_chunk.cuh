// Attention for many query rows per key head: bound by the products, on tcgen05.
//
// A unit is 256 packed rows (attn_units.cuh), as two tiles of 128 rows.  One CTA per SM:
//   warps 0-3, 4-7   softmax of row tile 0 and 1, one row a thread;
//   warps 8-11       loads: queries, keys and values from their pages, by cp.async into the
//                    128-byte swizzled layout that the matrix instructions read.  Page
//                    boundaries may fall anywhere in a tile and slots past the length are
//                    filled with zeros, which a box copy could do neither of;
//   warp 12          issues the products;
//   warp 13          hands what the load warps wrote over to the tensor cores' proxy
//                    (14 and 15 make the warpgroup whole).
// S = Q K^T goes to tensor memory (128 columns a tile), the softmax warps read it, write the
// weights P over it in the input type, and O += P V takes P from there: scores never touch
// shared memory.  The two tiles alternate: while one is in its softmax, the tensor cores
// have the other's PV and next QK^T (2 x 128 x 128 x D each).  O stays in tensor memory;
// it is rescaled only when a row's maximum has grown by more than 2^8 since the last
// time (P and its sum are then up to 2^8, which both types hold), so hardly ever.
// A unit of at most 128 rows has one row tile: both halves of the CTA then take the same
// queries and every other key tile, and their sums are joined like those of two spans.
#pragma once

#include <type_traits>

#include "attn_stream.cuh"
#include "tcgen05.cuh"

namespace clsample {

constexpr int kChunkThreads = 512;
constexpr int kChunkRows = 256;
constexpr int kChunkKeys = 128;
constexpr float kRescaleAt = 8.f;  // log2

// Registers a thread by warpgroup: 2 x softmax, loads, products.  They add up to what the
// block is launched with (4 x 128).
constexpr int kSoftmaxRegs = 176, kLoadRegs = 80, kMmaRegs = 80;
static_assert(2 * kSoftmaxRegs + kLoadRegs + kMmaRegs == 4 * (65536 / kChunkThreads), "the launch's registers");

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Two float32 operations in one instruction.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split_pair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <int D>
struct ChunkShape {
  static constexpr int kKeySlots = D == 128 ? 2 : 4;  // ring of key tiles
  static constexpr int kValueSlots = kKeySlots + 1;   // values are needed a step later
  static constexpr int kTile = 128 * D * 2;           // 128 rows, in bytes
  static constexpr int kBytes = (2 + kKeySlots + kValueSlots) * kTile + 1024;  // 1024: alignment of the swizzle
};

template <int NS, int NV>
struct ChunkShared {
  // filled by the load warps; handed over; S of a tile complete, so that its keys' slot and
  // the slot of the values before them are free
  unsigned long long k_landed[NS], v_landed[NV], k_full[NS], v_full[NV], tile_done[NS];
  unsigned long long q_full, q_empty, end, s_full[2], p_half[2], p_full[2], o_full[2];
  uint32_t tmem;
  volatile int dead;           // a bounded wait ran out: every other wait ends too
  uint32_t key_ok[2 * NS][4];  // keys of a tile that are on valid pages
};

// Bounded wait for a phase: about two seconds, then the CTA gives up.
__device__ __forceinline__ bool chunk_wait(unsigned long long* bar, uint32_t parity, volatile int* dead) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long start = clock64();
  for (uint32_t i = 1; i < kSpinLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 0 && (*dead || clock64() - start > 4000000000ll)) break;
  }
  *dead = 1;
  return false;
}

// Bits lo .. hi of a word, of which only 0 .. 31 exist.
__device__ __forceinline__ uint32_t column_bits(int lo, int hi) {
  const uint32_t upto = hi >= 31 ? ~0u : hi < 0 ? 0u : (2u << hi) - 1;
  return lo <= 0 ? upto : lo > 31 ? 0u : upto & (~0u << lo);
}

struct SoftmaxSync {  // the 256 softmax threads
  static __device__ __forceinline__ void sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
};

// Joins the parts of a unit, as join_parts does, by the 256 softmax threads.  A slot holds
// four sums of each row side by side, then the next four of each row, so that threads with a
// row each read and write whole lines.  With `split` a CTA's part is two, 128 rows apart, and
// two threads share a row.
template <class T, int D>
__device__ __forceinline__ void join_rows(const AttnParams& P, const Unit& u, const Span& span, int64_t unit_begin,
                                          bool split) {
  __shared__ int last;
  const int tid = threadIdx.x;
  const int c0 = cta_of_tile(span, unit_begin), c1 = cta_of_tile(span, unit_begin + u.tiles - 1);
  if (c0 < c1) {
    __threadfence();
    SoftmaxSync::sync();
    if (tid == 0) {
      last = atomicAdd(P.arrived + c0, 1) == c1 - c0;
      if (last) P.arrived[c0] = 0;  // for the next call
    }
    SoftmaxSync::sync();
    if (!last) return;
    __threadfence();
  } else {
    SoftmaxSync::sync();  // only this CTA's own two halves
  }
  const int halves = split ? 2 : 1, parts = (c1 - c0 + 1) * halves;
  const int r = split ? tid & 127 : tid;
  const int d0 = split ? (tid >> 7) * (D / 2) : 0, d1 = split ? d0 + D / 2 : D;
  auto slot_of = [&](int part) {
    const int c = c0 + part / halves;
    return scratch_slot<kChunkRows, D>(P, c, c == c0 ? 1 : 0);
  };
  if (r < u.rows) {
    float m = __int_as_float(0xff800000), l = 0.f;
    for (int part = 0; part < parts; ++part) {
      const float* s = slot_of(part) + kChunkRows * D + r + (part % halves) * 128;
      const float mc = __ldcg(s), lc = __ldcg(s + kChunkRows);
      const float mn = fmaxf(m, mc);
      l = l * (m == mn ? 1.f : exp2_fast(m - mn)) + lc * (mc == mn ? 1.f : exp2_fast(mc - mn));
      m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int row = u.row0 + r;
    T* dst = (T*)P.a.out + (int64_t)(u.q0 + row / P.g) * P.a.o_stride_t +
             (int64_t)(u.h * P.g + row % P.g) * P.a.o_stride_h;
    if (d0 == 0) store_lse(P, u, r, m, l);
    for (int d = d0; d < d1; d += 32) {
      float4 o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int part = 0; part < parts; ++part) {
        const float* s = slot_of(part);
        const int at = r + (part % halves) * 128;
        const float mc = __ldcg(s + kChunkRows * D + at);
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = __ldcg(reinterpret_cast<const float4*>(s + (d + 4 * i) * kChunkRows + at * 4));
        const float f = (mc == m ? 1.f : exp2_fast(mc - m)) * inv;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = make_float4(fmaf(v[i].x, f, o[i].x), fmaf(v[i].y, f, o[i].y), fmaf(v[i].z, f, o[i].z),
                             fmaf(v[i].w, f, o[i].w));
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        *reinterpret_cast<uint4*>(dst + d + 4 * i) =
            make_uint4(Pair<T>::narrow(o[i].x, o[i].y), Pair<T>::narrow(o[i].z, o[i].w),
                       Pair<T>::narrow(o[i + 1].x, o[i + 1].y), Pair<T>::narrow(o[i + 1].z, o[i + 1].w));
    }
  }
  if (split) SoftmaxSync::sync();  // the CTA may write the same slot for its next unit
}

template <class T, int D>
__global__ void __launch_bounds__(kChunkThreads, 1) attn_chunk_kernel(const __grid_constant__ AttnParams P) {
  using Shape = ChunkShape<D>;
  constexpr int NS = Shape::kKeySlots, NV = Shape::kValueSlots, kTile = Shape::kTile, KC = D / 8;
  constexpr int kHalf = 128 * 128;  // bytes of 128 rows of 64 elements
  extern __shared__ unsigned char raw[];
  __shared__ ChunkShared<NS, NV> sh;
  unsigned char* const smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t q_smem = smem_addr(smem), k_smem = q_smem + 2 * kTile, v_smem = k_smem + NS * kTile;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const clsample_attention_args_t& a = P.a;
  const float neg_inf = __int_as_float(0xff800000);

  if (a.row_status) attention_status<kChunkThreads>(P);
  Span span;
  Unit u;
  int64_t unit_begin;
  if (!find_span<kChunkRows, kChunkKeys, kChunkThreads>(P, &span, &u, &unit_begin)) return;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sh.k_landed[i], 128 + 4);  // every load thread's copies, and four words of key_ok
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.tile_done[i], 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(&sh.v_landed[i], 128);
      mbar_init(&sh.v_full[i], 1);
    }
    mbar_init(&sh.q_full, 128);
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.end, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&sh.s_full[w], 1);
      mbar_init(&sh.p_half[w], 4);
      mbar_init(&sh.p_full[w], 4);
      mbar_init(&sh.o_full[w], 1);
    }
    sh.dead = 0;
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc512(&sh.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  int64_t t = span.t0;

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax
    regs_up<kSoftmaxRegs>();
    const int w = warp >> 2;
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;  // 32 lanes a warp, lane in bits 16..
    const uint32_t s_tmem = tmem + lane_base + w * 128, o_tmem = tmem + lane_base + 256 + w * 128;
    uint32_t s_phase = 0, o_phase = 0, tile = 0;
    while (true) {
      const int j0 = (int)(t - unit_begin);
      const int cnt = (int)min((int64_t)(u.tiles - j0), span.t1 - t);
      const bool split = u.rows <= 128;  // this half has the key tiles w, w + 2, ..
      const bool done = cnt == u.tiles && !split;
      const int step = split ? 2 : 1;
      const int place = w * 128 + (warp & 3) * 32 + lane;  // of this row's sums in the scratch
      const int r = split ? place & 127 : place;
      if (!split || cnt > w) {
        const bool live = r < u.rows;
        const int first_pos = u.len - u.n;
        const int pos = live ? first_pos + (u.row0 + r) / P.g : -1;
        const int half0 = split ? 0 : w * 128;
        const int pos_first = first_pos + (u.row0 + half0) / P.g;
        const int pos_last = first_pos + (u.row0 + min(u.rows, half0 + 128) - 1) / P.g;
        float m = neg_inf, l = 0.f;  // reference maximum (log2 units) and weights' sum
        const int jw = split ? w : 0;
        for (int j = jw; j < cnt; j += step) {
          const int kb = (u.tile0 + j0 + j) * kChunkKeys;
          if (lane == 0) {
            chunk_wait(&sh.s_full[w], s_phase, &sh.dead);
            // S of the tile's last half is complete
            if ((warp & 3) == 0 && (split || w == 1)) mbar_arrive(&sh.tile_done[(tile + j) % NS]);
          }
          __syncwarp();
          s_phase ^= 1;
          tc_fence_after();
          const uint32_t* ok = sh.key_ok[(tile + j) % (2 * NS)];
          const uint32_t ok0 = ok[0], ok1 = ok[1], ok2 = ok[2], ok3 = ok[3];
          const bool whole = (ok0 & ok1 & ok2 & ok3) == ~0u && kb + 127 <= pos_first &&
                             (a.window <= 0 || kb > pos_last - a.window);
          uint32_t x[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(*reinterpret_cast<uint32_t(*)[32]>(x + c * 32), s_tmem + c * 32);
          tmem_wait_ld();
          if (!whole) {
            const int hi = pos - kb;  // columns lo .. hi are seen
            const int lo = a.window > 0 ? hi - a.window + 1 : 0;
            const uint32_t shown[4] = {ok0 & column_bits(lo, hi), ok1 & column_bits(lo - 32, hi - 32),
                                       ok2 & column_bits(lo - 64, hi - 64), ok3 & column_bits(lo - 96, hi - 96)};
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (!(shown[c >> 5] & (1u << (c & 31)))) x[c] = 0xff800000u;
          }
          float tops[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) tops[i] = fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 4]));
#pragma unroll
          for (int c = 8; c < 128; c += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              tops[i] = max3(tops[i], __uint_as_float(x[c + i]), __uint_as_float(x[c + 4 + i]));
          const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * P.scale_log2;
          const bool grow = top > m + kRescaleAt || (m == neg_inf && top > neg_inf);
          if (__any_sync(~0u, grow)) {
            const float keep = grow ? exp2_fast(m - top) : 1.f;
            if (grow) m = top;
            l *= keep;
            if (j > jw) {
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                uint32_t y[16];
                tmem_ld16(y, o_tmem + c * 16);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * keep);
                tmem_st16(o_tmem + c * 16, y);
              }
            }
          }
          const float base = m == neg_inf ? 0.f : -m;
          const uint64_t scale2 = pair_of(P.scale_log2, P.scale_log2), base2 = pair_of(base, base);
          uint64_t sums[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int i = c * 32 + 2 * e;
              const float2 y = split_pair(fma2(pair_of(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), scale2, base2));
              const float p0 = exp2_fast(y.x), p1 = exp2_fast(y.y);
              sums[e & 1] = add2(sums[e & 1], pair_of(p0, p1));
              p[e] = Pair<T>::narrow(p0, p1);
            }
            tmem_st16(s_tmem + c * 16, p);
            if (c & 1) {  // the product starts on the first 64 keys
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(c == 1 ? &sh.p_half[w] : &sh.p_full[w]);
            }
          }
          const float2 s0 = split_pair(add2(sums[0], sums[1]));
          l += s0.x + s0.y;
        }
        chunk_wait(&sh.o_full[w], o_phase, &sh.dead);
        o_phase ^= 1;
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float* slot = scratch_slot<kChunkRows, D>(P, blockIdx.x, j0 == 0 ? 1 : 0);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[32];
          tmem_ld32(x, o_tmem + c * 32);
          tmem_wait_ld();
          if (live) {
            if (done) {
              T* dst = (T*)a.out + (int64_t)(u.q0 + (u.row0 + r) / P.g) * a.o_stride_t +
                       (int64_t)(u.h * P.g + (u.row0 + r) % P.g) * a.o_stride_h + c * 32;
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  y[i] = l == 0.f ? 0u
                                  : Pair<T>::narrow(__uint_as_float(x[e + 2 * i]) * inv,
                                                    __uint_as_float(x[e + 2 * i + 1]) * inv);
                *reinterpret_cast<uint4*>(dst + e) = make_uint4(y[0], y[1], y[2], y[3]);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                __stcg(reinterpret_cast<uint4*>(slot + ((c * 32 + e) * kChunkRows + place * 4)),
                       make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]));
            }
          }
        }
        tc_fence_before();  // O has been read: the next unit's products may overwrite it
        if (live) {
          if (done) {
            store_lse(P, u, r, m, l);
          } else {
            __stcg(slot + kChunkRows * D + place, m);
            __stcg(slot + kChunkRows * D + kChunkRows + place, l);
          }
        }
      } else if (r < u.rows) {  // no key tile for this half
        float* slot = scratch_slot<kChunkRows, D>(P, blockIdx.x, j0 == 0 ? 1 : 0);
        for (int d = 0; d < D; d += 4)
          __stcg(reinterpret_cast<float4*>(slot + (d * kChunkRows + place * 4)), make_float4(0.f, 0.f, 0.f, 0.f));
        __stcg(slot + kChunkRows * D + place, neg_inf);
        __stcg(slot + kChunkRows * D + kChunkRows + place, 0.f);
      }
      if (!done) join_rows<T, D>(P, u, span, unit_begin, split);
      if (sh.dead && tid == 0 && a.row_status) atomicMax(a.row_status + u.b, CLSAMPLE_ROW_OVERFLOW);
      tile += cnt;
      t += cnt;
      if (t >= span.t1) break;
      unit_begin = t;
      next_unit<kChunkRows, kChunkKeys>(P, &u);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ loads
    regs_down<kLoadRegs>();
    const int lw = warp - 8;
    uint32_t it = 0, seg = 0;
    while (true) {
      const int j0 = (int)(t - unit_begin);
      const int cnt = (int)min((int64_t)(u.tiles - j0), span.t1 - t);
      chunk_wait(&sh.q_empty, (seg & 1) ^ 1, &sh.dead);
#pragma unroll 1
      for (int w = 0; w < 2; ++w) {
        const int mine = u.row0 + w * 128 + lw * 32 + lane;  // this lane's row, which it hands to the others
        const bool live = mine < u.row0 + u.rows;
        const int64_t off = live ? (int64_t)(u.q0 + mine / P.g) * a.q_stride_t +
                                       (int64_t)(u.h * P.g + mine % P.g) * a.q_stride_h
                                 : 0;
        const unsigned mask = __ballot_sync(~0u, live);
#pragma unroll
        for (int x = 0; x < KC; ++x) {
          const int i = x * 32 + lane, row = i / KC, ch = i % KC, r = lw * 32 + row;
          const int64_t o = __shfl_sync(~0u, off, row) + ch * 8;
          cp_async16(q_smem + w * kTile + (ch >> 3) * kHalf + r * 128 + (((ch & 7) ^ (r & 7)) << 4),
                     (const T*)a.q + o, (mask >> row) & 1);
        }
      }
      cp_async_arrive(smem_addr(&sh.q_full));
      const T* kc = (const T*)a.k_cache + (int64_t)u.h * a.head_stride;
      const T* vc = (const T*)a.v_cache + (int64_t)u.h * a.head_stride;
      const int32_t* table = a.page_table + (int64_t)u.b * a.table_stride;
      auto page_of = [&](int j) {
        const int key = (u.tile0 + j0 + j) * kChunkKeys + lw * 32 + lane;
        if (j >= cnt || key < u.key_lo || key >= u.key_hi) return -1;
        const int id = __ldg(table + (P.page_shift >= 0 ? key >> P.page_shift : key / a.page_size));
        return id < a.num_pages ? id : -1;
      };
      int page = page_of(0);
      for (int j = 0; j < cnt; ++j, ++it) {
        const int next = page_of(j + 1);
        const int key = (u.tile0 + j0 + j) * kChunkKeys + lw * 32 + lane;
        const int slot = P.page_shift >= 0 ? key & ((1 << P.page_shift) - 1) : key % a.page_size;
        const bool ok = page >= 0;
        const int64_t off = ok ? (int64_t)page * a.page_stride + (int64_t)slot * a.slot_stride : 0;
        const unsigned mask = __ballot_sync(~0u, ok);
        // keys outside the unit's range are hidden by the rows' limits: only a bad page counts
        const unsigned shown = __ballot_sync(~0u, ok || key < u.key_lo || key >= u.key_hi);
        // the slot of the keys is free when S of the tile that had it is complete, and the slot
        // of the values when O is, which a later tile's completion covers: the next one's if
        // both halves take each tile, the one after it otherwise (and across units, where
        // either may have been the case)
        const int64_t k_gate = (int64_t)it - NS, v_gate = (int64_t)it - NV + (u.rows <= 128 || j < NV ? 2 : 1);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          const int64_t gate = kv ? v_gate : k_gate;
          // (the keys' gate has been passed: by now its barrier may be a phase further)
          if (gate >= 0 && (kv == 0 || v_gate > k_gate)) chunk_wait(&sh.tile_done[gate % NS], (gate / NS) & 1, &sh.dead);
          __syncwarp();
          unsigned long long* landed = kv ? &sh.v_landed[it % NV] : &sh.k_landed[it % NS];
          if (kv == 0 && lane == 0) {
            sh.key_ok[it % (2 * NS)][lw] = shown;
            mbar_arrive(landed);
          }
          const T* src = kv ? vc : kc;
          const uint32_t dst = kv ? v_smem + it % NV * kTile : k_smem + it % NS * kTile;
#pragma unroll
          for (int x = 0; x < KC; ++x) {
            const int i = x * 32 + lane, row = i / KC, ch = i % KC, r = lw * 32 + row;
            const int64_t o = __shfl_sync(~0u, off, row) + ch * 8;
            cp_async16(dst + (ch >> 3) * kHalf + r * 128 + (((ch & 7) ^ (r & 7)) << 4), src + o, (mask >> row) & 1);
          }
          cp_async_arrive(smem_addr(landed));
        }
        page = next;
      }
      ++seg;
      t += cnt;
      if (t >= span.t1) break;
      unit_begin = t;
      next_unit<kChunkRows, kChunkKeys>(P, &u);
    }
    cp_async_wait_all();
  } else {
    // ------------------------------------------------------------------ products
    regs_down<kMmaRegs>();
    if (warp == 12) {
      // Everything here is uniform, and made known as such (uni): the operands of a product
      // have to be in uniform registers for the issue to keep up with the tensor cores.
      auto uni = [](uint32_t x) { return __shfl_sync(~0u, x, 0); };
      constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
      constexpr uint32_t kQk = f16_idesc(kBf16, 128, 128, false), kPv = f16_idesc(kBf16, 128, D, true);
      const uint32_t base = uni(tmem), q_desc = uni(smem_desc_lo(q_smem, 16)), k_desc = uni(smem_desc_lo(k_smem, 16)),
                     v_desc = uni(smem_desc_lo(v_smem, kHalf));
      uint32_t it = 0, seg = 0, p_phase = 0;  // bit w of p_phase: half w
      bool alive = true;
      auto wait = [&](unsigned long long* bar, uint32_t parity) {
        alive = __all_sync(~0u, chunk_wait(bar, parity, &sh.dead)) && alive;
      };
      auto keys_ready = [&](uint32_t tile) { wait(&sh.k_full[tile % NS], (tile / NS) & 1); };
      auto values_ready = [&](uint32_t tile) { wait(&sh.v_full[tile % NV], (tile / NV) & 1); };
      // S of half w = (row tile rt of Q) K^T
      auto qk = [&](uint32_t w, uint32_t rt, uint32_t tile) {
        const uint32_t q0 = q_desc + rt * (kTile >> 4), k0 = k_desc + (tile % NS) * (kTile >> 4);
        if (alive) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
            mma_ss(base + w * 128, q0 + off, k0 + off, kQk, ks > 0);
          }
        }
        mma_commit(&sh.s_full[w]);
      };
      // O of half w (+)= P V, in two parts as P comes
      auto pv = [&](uint32_t w, uint32_t tile, bool add) {
        const uint32_t v0 = v_desc + (tile % NV) * (kTile >> 4), o = base + 256 + w * 128, p0 = base + w * 128;
        const uint32_t parity = (p_phase >> w) & 1;
        const bool all = __all_sync(~0u, mbar_test_wait(&sh.p_full[w], parity));
        if (!all) wait(&sh.p_half[w], parity);
        tc_fence_after();
        if (alive) {
          mma_ts(o, p0, v0, kPv, add);
#pragma unroll
          for (int ks = 1; ks < 4; ++ks) mma_ts(o, p0 + ks * 8, v0 + ks * (2048 >> 4), kPv, true);
        }
        if (!all) wait(&sh.p_full[w], parity);
        tc_fence_after();
        if (alive) {
#pragma unroll
          for (int ks = 4; ks < 8; ++ks) mma_ts(o, p0 + ks * 8, v0 + ks * (2048 >> 4), kPv, true);
        }
        p_phase ^= 1u << w;
      };
      while (true) {
        const int j0 = (int)(t - unit_begin);
        const int cnt = (int)uni((uint32_t)min((int64_t)(u.tiles - j0), span.t1 - t));
        const bool split = uni(u.rows <= 128);
        wait(&sh.q_full, seg & 1);
        fence_async_proxy();  // the copies were ordinary writes; the products read by the async proxy
        keys_ready(it);
        if (!split) {
          qk(0, 0, it);
          qk(1, 1, it);
          if (cnt == 1) mma_commit(&sh.q_empty);
          for (int j = 0; j + 1 < cnt; ++j, ++it) {
            keys_ready(it + 1);  // handed over after the values of tile it
            pv(0, it, j > 0);
            qk(0, 0, it + 1);
            pv(1, it, j > 0);
            qk(1, 1, it + 1);
          }
          if (cnt > 1) mma_commit(&sh.q_empty);
          values_ready(it);
          pv(0, it, cnt > 1);
          mma_commit(&sh.o_full[0]);
          pv(1, it, cnt > 1);
          mma_commit(&sh.o_full[1]);
          ++it;
        } else {
          qk(0, 0, it);
          if (cnt > 1) {
            keys_ready(it + 1);
            qk(1, 0, it + 1);
          }
          if (cnt <= 2) mma_commit(&sh.q_empty);
          for (int j = 0; j < cnt; ++j, ++it) {
            const uint32_t w = j & 1;
            values_ready(it);
            pv(w, it, j > 1);
            if (j + 2 < cnt) {
              keys_ready(it + 2);
              qk(w, 0, it + 2);
              if (j + 3 == cnt) mma_commit(&sh.q_empty);
            } else {
              mma_commit(&sh.o_full[w]);
            }
          }
        }
        ++seg;
        t += cnt;
        if (uni(t >= span.t1)) break;
        unit_begin = t;
        next_unit<kChunkRows, kChunkKeys>(P, &u);
      }
      // products still running when a wait gave up end before their memory is freed
      if (!alive) {
        mma_commit(&sh.end);
        for (int i = 0; i < 1 << 16 && !mbar_try_wait(&sh.end, 0); ++i) __nanosleep(100);
      }
    } else if (warp == 13 && lane == 0) {
      // The copies are ordinary writes, the products read by the async proxy: the fence between
      // them costs a hundred cycles or so, which the issuing warp has not got.
      const int tiles = (int)(span.t1 - span.t0);
      for (int i = 0; i < tiles; ++i) {
        chunk_wait(&sh.k_landed[i % NS], (i / NS) & 1, &sh.dead);
        fence_async_proxy();
        mbar_arrive(&sh.k_full[i % NS]);
        chunk_wait(&sh.v_landed[i % NV], (i / NV) & 1, &sh.dead);
        fence_async_proxy();
        mbar_arrive(&sh.v_full[i % NV]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_free512(tmem);
}

}  // namespace clsample
