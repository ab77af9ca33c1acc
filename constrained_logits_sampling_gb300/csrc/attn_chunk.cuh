// Attention for many query rows per key head: bound by the products, on tcgen05.
//
// A unit is 256 packed rows (attn_units.cuh), as two tiles of 128 rows.  One CTA per SM:
//   warps 0-3, 4-7   softmax of row tile 0 and 1, one row a thread;
//   warps 8, 9, 11   loads (below);
//   warp 10          issues the products.
// Loads come in two forms.  Where pages are whole boxes of a tile (8, 16, 32, 64 or a
// multiple of 128 slots) warps 8 and 11 copy keys and values by TMA, one box a page and 64
// elements, an invalid page as zeros (a box takes some 75 cycles to issue, so with pages of 16
// slots one warp would not keep up: on an earlier version 771 us against 574); warp 9 loads the
// queries, in one box a row tile where the query heads of a key head divide 128 and row by row
// otherwise, and clears the value slots that lie outside the unit's keys (they may hold anything,
// and 0 x NaN is NaN).
// Other page sizes are copied row by row with cp.async by warps 8 and 9, zeros where there
// is no key, and warp 11 hands what has landed over to the tensor cores' proxy.
// S = Q K^T goes to tensor memory (128 columns a tile), the softmax warps read it, write the
// weights P over it in the input type, and O += P V takes P from there: scores never touch
// shared memory.  The two tiles alternate: while one is in its softmax, the tensor cores
// have the other's PV and next QK^T (2 x 128 x 128 x D each).  O stays in tensor memory;
// it is rescaled only when a row's maximum has grown by more than 2^8 since the last
// time (P and its sum are then up to 2^8, which both types hold), so hardly ever.
// 2 x 2048 tokens on 32 / 8 heads of 128 over 14500 to 15600 keys (943 GFLOP): 561 us a call with
// L2 flushed in between (1.68 PFLOP/s), 615 to 635 in a row of calls that draw the power limit.
// The products of a tile of 128 keys take 2048 cycles; a trace of an earlier version showed about
// 2500 a tile, the rest of it the way from a finished S over the softmax (970) to the next product.
// A unit of at most 128 rows has one row tile: both halves of the CTA then take the same
// queries and every other key tile, and their sums are joined at the end, in the room of the
// second row tile's queries.
#pragma once

#include <type_traits>

#include "attn_stream.cuh"
#include "tcgen05.cuh"

namespace clsample {

constexpr int kChunkThreads = 384;
constexpr int kChunkRows = 256;
constexpr int kChunkKeys = 128;
constexpr float kRescaleAt = 8.f;  // log2

// Registers a thread: the two softmax warpgroups, and the one of loads and products.  They
// add up to what the block is launched with (3 x 168).
constexpr int kSoftmaxRegs = 200, kOtherRegs = 104;
static_assert(2 * kSoftmaxRegs + kOtherRegs == 3 * 168 && 168 * kChunkThreads <= 65536, "the launch's registers");

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
  unsigned long long k_landed[NS], v_landed[NV], k_full[NS], v_full[NV], tile_done[2 * NS];
  unsigned long long q_full, q_empty, end, s_full[2], p_half[2], p_full[2], o_full[2];
  unsigned long long unit_full[2], unit_done[2];  // of the units with even and odd numbers
  uint32_t tmem;
  // The units that the softmax warps are at, by the load warps, which are ahead: those have no
  // registers to spare for more than they need at a time.
  Unit unit[2];
  int64_t unit_begin[2];
  Span span;
  WaitLimit limit;
  alignas(16) uint32_t key_ok[2 * NS][4];  // keys of a tile that are on valid pages
};

// Bits lo .. hi of a word, of which only 0 .. 31 exist.
__device__ __forceinline__ uint32_t column_bits(int lo, int hi) {
  const uint32_t upto = hi >= 31 ? ~0u : hi < 0 ? 0u : (2u << hi) - 1;
  return lo <= 0 ? upto : lo > 31 ? 0u : upto & (~0u << lo);
}

struct SoftmaxSync {  // the 256 softmax threads
  static __device__ __forceinline__ void sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
  static __device__ __forceinline__ bool all(bool yes) {  // and whether all of them say yes
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)yes)
        : "memory");
    return r != 0;
  }
};

// How a CTA ends when a wait has run out, so that nothing is left waiting or in flight and every
// address stays one of the call's.  The wait's thread marks the CTA dead before it goes on, on
// whatever is there.  Who waits for that one's arrivals goes on too, so the load warps look at the
// mark after each wait: they announce and make no more copies, hand over no more units, and leave
// after the unit that they have.  The warp of products issues none after a wait of its own that
// failed.  The softmax threads finish the unit that they have, as its barriers take all 256 of
// them, and go on to no other.  Then all pause while copies land.  The call's statuses tell that
// its outputs are void.

template <class T, int D, bool kTma>
__global__ void __launch_bounds__(kChunkThreads, 1)
    attn_chunk_kernel(const __grid_constant__ AttnParams P, const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap q_map) {
  using Shape = ChunkShape<D>;
  constexpr int NS = Shape::kKeySlots, NV = Shape::kValueSlots, kTile = Shape::kTile, KC = D / 8;
  constexpr int kHalf = 128 * 128;  // bytes of 128 rows of 64 elements
  constexpr int kRowWarps = kTma ? 1 : 2;  // that copy rows
  extern __shared__ unsigned char raw[];
  __shared__ ChunkShared<NS, NV> sh;
  unsigned char* const smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t q_smem = smem_addr(smem), k_smem = q_smem + 2 * kTile, v_smem = k_smem + NS * kTile;
  // The warp's number is made known as uniform, as its role's branches are: without it 2 x 1024 tokens
  // over 7100 keys took 177 us instead of 157.
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  const clsample_attention_args_t& a = P.a;
  const float neg_inf = __int_as_float(0xff800000);

  let_next_grid_start();
  Span span;
  Unit u;
  int64_t unit_begin;
  if (!find_span<kChunkRows, kChunkKeys, kChunkThreads>(P, &span, &u, &unit_begin)) {
    if (tid == 0) P.cut[blockIdx.x].rows = 0;
    return;
  }

  if (tid == 0) {
    // for tests: a barrier that waits for one arrival more than it gets
    auto init = [&](unsigned long long* bar, int count, int stall, int slot = 0) {
      mbar_init(bar, count + (P.stall == (stall << 8) + slot ? 1 : 0));
    };
    for (int i = 0; i < NS; ++i) {
      init(&sh.k_landed[i], 64 + 2, kStallKeysLanded, i);  // every load thread's copies, and each warp's words of key_ok
      init(&sh.k_full[i], 1, kStallKeys, i);
      init(&sh.tile_done[i], 1, kStallTileDone, i);
      init(&sh.tile_done[NS + i], 1, kStallTileDone, NS + i);
    }
    for (int i = 0; i < NV; ++i) {
      init(&sh.v_landed[i], kTma ? 1 : 64, kStallValuesLanded, i);
      init(&sh.v_full[i], 1, kStallValues, i);
    }
    init(&sh.q_full, kTma && P.q_box ? 1 : 32 * kRowWarps, kStallQueries);
    init(&sh.q_empty, 1, kStallQueriesDone);
    mbar_init(&sh.end, 1);
    for (int w = 0; w < 2; ++w) {
      init(&sh.s_full[w], 1, kStallScores, w);
      init(&sh.p_half[w], 4, kStallHalfWeights, w);
      init(&sh.p_full[w], 4, kStallWeights, w);
      init(&sh.o_full[w], 1, kStallSums, w);
      init(&sh.unit_full[w], 1, kStallUnit, w);
      init(&sh.unit_done[w], 1, kStallUnitDone, w);
    }
    sh.limit.cycles = P.wait_cycles;
    sh.limit.dead = 0;
    sh.span = span;
    fence_mbar_init();
  }
  if (warp == 10) tmem_alloc512(&sh.tmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  int64_t t = span.t0;

  // A whole warpgroup has to run the same register instruction, so warps 8 to 11 do before they part.
  if (warp >= 8) regs_down<kOtherRegs>();
  if (warp < 8) {
    // ------------------------------------------------------------------ softmax
    regs_up<kSoftmaxRegs>();
    const int w = warp >> 2;
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;  // 32 lanes a warp, lane in bits 16..
    const uint32_t s_tmem = tmem + lane_base + w * 128, o_tmem = tmem + lane_base + 256 + w * 128;
    uint32_t s_phase = 0, o_phase = 0, tile = 0;
    bool noted = false, go = SoftmaxSync::all(bounded_wait(&sh.unit_full[0], 0, &sh.limit));
    for (uint32_t seg = 0; go; ++seg) {
      const Unit& u = sh.unit[seg & 1];
      const int j0 = (int)max(sh.span.t0 - sh.unit_begin[seg & 1], (int64_t)0);
      const int cnt = (int)(min(sh.unit_begin[seg & 1] + u.tiles, sh.span.t1) - sh.unit_begin[seg & 1]) - j0;
      const bool split = u.rows <= 128;  // this half has the key tiles w, w + 2, ..
      const int step = split ? 2 : 1, jw = split ? w : 0;
      const int r = (split ? 0 : w * 128) + (warp & 3) * 32 + lane;  // this thread's row
      const bool live = r < u.rows;
      float m = neg_inf, l = 0.f;  // reference maximum (log2 units) and weights' sum
      if (cnt > jw) {
        const int first_pos = u.len - u.n, kb0 = (u.tile0 + j0) * kChunkKeys;
        const int pos = live ? first_pos + token_of(P, u.row0 + r) : -1;
        const int half0 = split ? 0 : w * 128;
        const int pos_first = first_pos + token_of(P, u.row0 + half0);
        const int pos_last = first_pos + token_of(P, u.row0 + min(u.rows, half0 + 128) - 1);
        for (int j = jw; j < cnt; j += step) {
          const int kb = kb0 + j * kChunkKeys;
          bounded_wait(&sh.s_full[w], s_phase, &sh.limit);
          if (lane == 0) {
            if ((warp & 3) == 0 && (split || w == 1)) mbar_arrive(&sh.tile_done[(tile + j) % (2 * NS)]);
          }
          __syncwarp();
          s_phase ^= 1;
          tc_fence_after();
          const uint32_t* ok = sh.key_ok[(tile + j) % (2 * NS)];
          const uint4 bits = *reinterpret_cast<const uint4*>(ok);
          const bool whole = (bits.x & bits.y & bits.z & bits.w) == ~0u && kb + 127 <= pos_first &&
                             (a.window <= 0 || kb > pos_last - a.window);
          uint32_t x[128];
          tmem_ld(x, s_tmem);
          if (!whole) {
            const int hi = pos - kb;  // columns lo .. hi are seen
            const int lo = a.window > 0 ? hi - a.window + 1 : 0;
            const uint32_t shown[4] = {bits.x & column_bits(lo, hi), bits.y & column_bits(lo - 32, hi - 32),
                                       bits.z & column_bits(lo - 64, hi - 64), bits.w & column_bits(lo - 96, hi - 96)};
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (!(shown[c >> 5] & (1u << (c & 31)))) x[c] = 0xff800000u;
          }
          // weights of columns c0 .. c0 + 63 against the reference maximum, and their sums
          const uint64_t scale2 = pair_of(P.scale_log2, P.scale_log2);
          uint32_t p[32];
          uint64_t sums[2];
          auto weights = [&](int c0) {
            const float base = m == neg_inf ? 0.f : -m;
            const uint64_t base2 = pair_of(base, base);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int i = c0 + 2 * e;
              const float2 y = split_pair(fma2(pair_of(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), scale2, base2));
              const float p0 = exp2_fast(y.x), p1 = exp2_fast(y.y);
              sums[e & 1] = add2(sums[e & 1], pair_of(p0, p1));
              p[e] = Pair<T>::narrow(p0, p1);
            }
          };
          auto hand_over = [&](int c0, unsigned long long* bar) {
            tmem_st32(s_tmem + c0 / 2, p);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
          };
          // The first half is computed before the tile's maximum is known, so that the two
          // overlap; where the maximum calls for another reference (hardly ever after a unit's
          // first tile), once more.
          while (true) {
            sums[0] = sums[1] = 0;
            weights(0);
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
            if (!__any_sync(~0u, grow)) break;
            const float keep = grow ? exp2_fast(m - top) : 1.f;
            if (grow) m = top;
            l *= keep;
            if (j > jw) {
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t y[16];
                tmem_ld(y, o_tmem + c * 16);
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * keep);
                tmem_st16(o_tmem + c * 16, y);
              }
            }
          }
          hand_over(0, &sh.p_half[w]);  // the product starts on the first 64 keys
          weights(64);
          hand_over(64, &sh.p_full[w]);
          const float2 s0 = split_pair(add2(sums[0], sums[1]));
          l += s0.x + s0.y;
        }
        bounded_wait(&sh.o_full[w], o_phase, &sh.limit);
        o_phase ^= 1;
        tc_fence_after();
      }
      // A slot of the scratch holds four sums of each row side by side, then the next four of
      // each row, so that threads with a row each write whole lines.
      float* slot = scratch_slot<kChunkRows, D>(P, blockIdx.x, j0 == 0 ? 1 : 0);
      const bool done = cnt == u.tiles;
      // kCols columns at a time.  Four lanes have four rows; each stores a quarter of the columns
      // of all four, so that a store is of four times as many bytes a row.
      constexpr int kCols = D / 4, kWords = kCols / 8;
      const int row = u.row0 + min(r, u.rows - 1);
      const int64_t dst = (int64_t)(u.q0 + token_of(P, row)) * a.o_stride_t +
                          (int64_t)(u.h * P.g + head_of(P, row)) * a.o_stride_h;
      // this thread's row's sums, from column c on
      auto put = [&](const uint32_t (&x)[kCols], int c) {
        if (done) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          uint32_t y[4][kWords];
#pragma unroll
          for (int i = 0; i < kCols / 2; ++i)
            y[i / kWords][i % kWords] = l == 0.f ? 0u
                                        : Pair<T>::narrow(__uint_as_float(x[2 * i]) * inv,
                                                          __uint_as_float(x[2 * i + 1]) * inv);
#pragma unroll
          for (int s = 1; s <= 2; s *= 2) {
            const bool upper = lane & s;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i & s) continue;
#pragma unroll
              for (int e = 0; e < kWords; ++e) {
                const uint32_t got = __shfl_xor_sync(~0u, upper ? y[i][e] : y[i + s][e], s);
                if (upper)
                  y[i][e] = got;
                else
                  y[i + s][e] = got;
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int64_t to = __shfl_sync(~0u, dst, (lane & ~3) + i);
            T* at = (T*)a.out + to + c + (lane & 3) * (2 * kWords);
            if ((r & ~3) + i >= u.rows) continue;
            if constexpr (kWords == 4)
              *reinterpret_cast<uint4*>(at) = make_uint4(y[i][0], y[i][1], y[i][2], y[i][3]);
            else
              *reinterpret_cast<uint2*>(at) = make_uint2(y[i][0], y[i][1]);
          }
        } else if (live) {
#pragma unroll
          for (int e = 0; e < kCols; e += 4)
            __stcg(reinterpret_cast<uint4*>(slot + (c + e) * kChunkRows + r * 4),
                   make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]));
        }
      };
      if (split) {
        // each half joins one half of the columns and hands the other its sums of the rest
        float* const x_smem = reinterpret_cast<float*>(smem + kTile);
        constexpr int kRoom = 128 * kCols;  // of a half
        static_assert(2 * kRoom * 4 == kTile, "the second row tile's queries");
        x_smem[w * 256 + r] = m;
        x_smem[w * 256 + 128 + r] = l;
        SoftmaxSync::sync();
        const float mo = x_smem[(1 - w) * 256 + r], lo = x_smem[(1 - w) * 256 + 128 + r];
        const float mn = fmaxf(m, mo);
        const float mine = m == mn ? 1.f : exp2_fast(m - mn), others = mo == mn ? 1.f : exp2_fast(mo - mn);
        l = l * mine + lo * others;
        m = mn;
        SoftmaxSync::sync();
#pragma unroll 1
        for (int c = 0; c < D / 2; c += kCols) {
          uint32_t x[kCols];
          __syncwarp();
          tmem_ld(x, o_tmem + (1 - w) * (D / 2) + c);
#pragma unroll
          for (int e = 0; e < kCols; e += 4)  // a half without a key tile has no sums
            *reinterpret_cast<uint4*>(x_smem + w * kRoom + e * 128 + r * 4) =
                cnt > w ? make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]) : make_uint4(0, 0, 0, 0);
          SoftmaxSync::sync();
          tmem_ld(x, o_tmem + w * (D / 2) + c);
#pragma unroll
          for (int e = 0; e < kCols; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(x_smem + (1 - w) * kRoom + e * 128 + r * 4);
            const float ov[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              x[e + i] = __float_as_uint((cnt > w ? __uint_as_float(x[e + i]) * mine : 0.f) + ov[i] * others);
          }
          put(x, w * (D / 2) + c);
          SoftmaxSync::sync();
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < D; c += kCols) {
          uint32_t x[kCols];
          __syncwarp();
          tmem_ld(x, o_tmem + c);
          put(x, c);
        }
      }
      if (live && (w == 0 || !split)) {
        if (done) {
          store_lse(P, u, r, m, l);
        } else {
          __stcg(slot + kChunkRows * D + r, m);
          __stcg(slot + kChunkRows * D + kChunkRows + r, l);
        }
      }
      tc_fence_before();  // O has been read: the next unit's products may overwrite it
      tile += cnt;
      const bool last = sh.unit_begin[seg & 1] + u.tiles >= sh.span.t1;
      if (last && tid == 0) {
        note_cut(P, sh.span, u, sh.unit_begin[seg & 1]);
        noted = true;
      }
      if (split) fence_async_proxy();  // the room may next be written by a box copy
      // (the next unit is published without this one's end)
      go = SoftmaxSync::all(!last && bounded_wait(&sh.unit_full[(seg + 1) & 1], ((seg + 1) >> 1) & 1, &sh.limit) &&
                            !sh.limit.dead);
      if (go && tid == 0) mbar_arrive(&sh.unit_done[seg & 1]);
    }
    if (tid == 0 && !noted) P.cut[blockIdx.x].rows = 0;  // what an earlier call left there is not joined
  } else if (warp != 10) {
    // ------------------------------------------------------------------ loads
    const int lw = kTma ? 0 : warp - 8;  // of the warps that copy rows
    bool met = false;                    // the last unit's halves met in the second row tile's room
    const int tiles = (int)(span.t1 - span.t0);
    // 32 rows to rows r0.. of a tile; lane i has the place of row i, bit i of `live` tells
    // whether it is read or zero
    auto copy_rows = [&](const T* src, int64_t off, unsigned live, uint32_t dst, int r0) {
#pragma unroll
      for (int x = 0; x < KC; ++x) {
        const int i = x * 32 + lane, row = i / KC, ch = i % KC, r = r0 + row;
        const int64_t o = __shfl_sync(~0u, off, row) + ch * 8;
        cp_async16(dst + (ch >> 3) * kHalf + r * 128 + (((ch & 7) ^ (r & 7)) << 4), src + o, (live >> row) & 1);
      }
    };
    auto copy_queries = [&](uint32_t seg) -> bool {
      constexpr int kBlocks = 8 / kRowWarps;
      const bool box = kTma && P.q_box;
      int64_t off[kBlocks];
      unsigned live[kBlocks];
      if (!box) {  // each lane finds the places of its rows, one of 32, before it has to wait
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          const int mine = (i * kRowWarps + lw) * 32 + lane, row = u.row0 + mine;
          off[i] = mine < u.rows ? (int64_t)(u.q0 + token_of(P, row)) * a.q_stride_t +
                                       (int64_t)(u.h * P.g + head_of(P, row)) * a.q_stride_h
                                 : 0;
          live[i] = __ballot_sync(~0u, mine < u.rows);
        }
      }
      // the unit's place is free when the softmax warps are done with the one before the last
      const bool free = seg < 2 || bounded_wait(&sh.unit_done[seg & 1], ((seg - 2) >> 1) & 1, &sh.limit);
      if (lw == 0 && lane == 0 && free && !sh.limit.dead) {
        sh.unit[seg & 1] = u;
        sh.unit_begin[seg & 1] = unit_begin;
        mbar_arrive(&sh.unit_full[seg & 1]);
      }
      bounded_wait(&sh.q_empty, (seg & 1) ^ 1, &sh.limit);
      if (__any_sync(~0u, sh.limit.dead)) return false;
      const int tiles_of_rows = u.rows <= 128 ? 1 : 2;
      auto second_tile = [&]() {
        if (met) bounded_wait(&sh.unit_done[(seg - 1) & 1], ((seg - 1) >> 1) & 1, &sh.limit);
        __syncwarp();
      };
      if (box) {
        // (rows past the sequence's are other sequences' or zero, and are not stored)
        if (lane == 0) mbar_arrive_expect_tx(&sh.q_full, tiles_of_rows * kTile);
        for (int w = 0; w < tiles_of_rows; ++w) {
          if (w == 1) second_tile();
          if (lane < D / 64 && !sh.limit.dead)
            tma_load3(q_smem + w * kTile + lane * kHalf, &q_map, lane * 64, u.h * P.g,
                      u.q0 + token_of(P, u.row0 + w * 128), &sh.q_full);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          const int first = (i * kRowWarps + lw) * 32;
          if (first >= 128 && tiles_of_rows == 1) break;
          if (i == kBlocks / 2) second_tile();
          if (first < u.rows) copy_rows((const T*)a.q, off[i], live[i], q_smem + (first >> 7) * kTile, first & 127);
        }
        cp_async_arrive(smem_addr(&sh.q_full));
      }
      met = u.rows <= 128;
      return true;
    };
    // The slot of a tile's keys is free when S of the tile that had it is complete, and the
    // slot of its values when O is, which a later tile's completion covers: the next one's if
    // both halves take each tile, the one after it otherwise (and across units, where either
    // may have been the case).  Of twice as many completions as there are key slots the one
    // waited for is still the last on its barrier.
    auto tile_done = [&](int64_t gate) {
      if (gate >= 0) bounded_wait(&sh.tile_done[gate % (2 * NS)], (gate / (2 * NS)) & 1, &sh.limit);
      __syncwarp();
    };
    auto key_slot = [&](uint32_t it) { tile_done((int64_t)it - NS); };
    auto value_slot = [&](uint32_t it, int j) { tile_done((int64_t)it - NV + (u.rows <= 128 || j < NV ? 2 : 1)); };
    // a tile with values outside the unit's keys
    auto edge = [&](int tile) { return tile * kChunkKeys < u.key_lo || tile * kChunkKeys + kChunkKeys > u.key_hi; };

    if (kTma && warp != 9) {
      // lane i has the i-th page (or 128 slots of one) of a tile; warp 8 the keys, 11 the values
      const bool keys = warp == 8;
      const CUtensorMap* map = keys ? &k_map : &v_map;
      const int box = min(a.page_size, kChunkKeys), boxes = kChunkKeys / box;
      uint32_t it = 0;
      while (true) {
        const int j0 = (int)(t - unit_begin);
        const int cnt = (int)min((int64_t)(u.tiles - j0), span.t1 - t);
        const int32_t* table = a.page_table + (int64_t)u.b * a.table_stride;
        auto page_of = [&](int j) {  // num_pages, which is out of bounds: zeros
          const int key = (u.tile0 + j0 + j) * kChunkKeys + lane * box;
          if (j >= cnt || lane >= boxes || key + box <= u.key_lo || key >= u.key_hi) return a.num_pages;
          const int id = __ldg(table + (P.page_shift >= 0 ? key >> P.page_shift : key / a.page_size));
          return id >= 0 && id < a.num_pages ? id : -1;
        };
        int page = page_of(0);
        for (int j = 0; j < cnt; ++j, ++it) {
          const int tile = u.tile0 + j0 + j;
          const int key = tile * kChunkKeys + lane * box;
          const int slot = a.page_size > kChunkKeys ? key % a.page_size : 0;
          const unsigned bad = __ballot_sync(~0u, page < 0);
          const int from = page < 0 ? a.num_pages : page;
          page = page_of(j + 1);
          unsigned long long* full;
          uint32_t dst;
          if (keys) {
            key_slot(it);
            if (lane < 4) {
              uint32_t word = ~0u;
              if (bad)
                for (int e = 0; e < 32; ++e)
                  if ((bad >> ((lane * 32 + e) / box)) & 1) word &= ~(1u << e);
              sh.key_ok[it % (2 * NS)][lane] = word;
            }
            full = &sh.k_full[it % NS];
            dst = k_smem + it % NS * kTile;
          } else {
            value_slot(it, j);
            full = edge(tile) ? &sh.v_landed[it % NV] : &sh.v_full[it % NV];
            dst = v_smem + it % NV * kTile;
          }
          const bool dead = sh.limit.dead;
          __syncwarp();
          if (lane == 0 && !dead) mbar_arrive_expect_tx(full, kTile);
          __syncwarp();
          if (lane < boxes && !dead)
            for (int x = 0; x < D / 64; ++x)
              tma_load4(dst + x * kHalf + lane * box * 128, map, x * 64, slot, u.h, from, full);
        }
        t += cnt;
        if (t >= span.t1 || __any_sync(~0u, sh.limit.dead)) break;
        unit_begin = t;
        next_unit<kChunkRows, kChunkKeys>(P, &u);
      }
    } else if (kTma) {
      uint32_t it = 0, seg = 0, edges[NV] = {};  // phases of v_landed
      while (true) {
        const int j0 = (int)(t - unit_begin);
        const int cnt = (int)min((int64_t)(u.tiles - j0), span.t1 - t);
        if (!copy_queries(seg)) break;
        for (int j = 0; j < cnt; ++j) {
          const int tile = u.tile0 + j0 + j;
          if (!edge(tile)) continue;
          const uint32_t st = (it + j) % NV;
          uint32_t parity = 0;
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (i == st) parity = edges[i]++ & 1;
          bounded_wait(&sh.v_landed[st], parity, &sh.limit);
          const bool dead = sh.limit.dead;
          __syncwarp();
          const int lo = u.key_lo - tile * kChunkKeys, hi = u.key_hi - tile * kChunkKeys;
          for (int i = lane; i < 128 * KC; i += 32) {  // a row's pieces may lie anywhere in it: all are cleared
            const int row = i / KC, ch = i % KC;
            if (row < lo || row >= hi)
              *reinterpret_cast<uint4*>(smem + (2 + NS + st) * kTile + (ch >> 3) * kHalf + row * 128 + (ch & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_async_proxy();
          __syncwarp();
          if (lane == 0 && !dead) mbar_arrive(&sh.v_full[st]);
        }
        it += cnt;
        ++seg;
        t += cnt;
        if (t >= span.t1) break;
        unit_begin = t;
        next_unit<kChunkRows, kChunkKeys>(P, &u);
      }
      cp_async_wait_all();
    } else if (warp < 10) {
      uint32_t it = 0, seg = 0;
      while (true) {
        const int j0 = (int)(t - unit_begin);
        const int cnt = (int)min((int64_t)(u.tiles - j0), span.t1 - t);
        if (!copy_queries(seg)) break;
        const T* kc = (const T*)a.k_cache + (int64_t)u.h * a.head_stride;
        const T* vc = (const T*)a.v_cache + (int64_t)u.h * a.head_stride;
        const int32_t* table = a.page_table + (int64_t)u.b * a.table_stride;
        // warp lw has keys 64 lw .. 64 lw + 63 of a tile, two a lane
        auto page_of = [&](int j, int half) {
          const int key = (u.tile0 + j0 + j) * kChunkKeys + lw * 64 + half * 32 + lane;
          if (j >= cnt || key < u.key_lo || key >= u.key_hi) return -1;
          const int id = __ldg(table + (P.page_shift >= 0 ? key >> P.page_shift : key / a.page_size));
          return id < a.num_pages ? id : -1;
        };
        int page[2] = {page_of(0, 0), page_of(0, 1)};
        for (int j = 0; j < cnt; ++j, ++it) {
          int64_t off[2];
          unsigned live[2], shown[2];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int key = (u.tile0 + j0 + j) * kChunkKeys + lw * 64 + half * 32 + lane;
            const int slot = P.page_shift >= 0 ? key & ((1 << P.page_shift) - 1) : key % a.page_size;
            const bool ok = page[half] >= 0;
            off[half] = ok ? (int64_t)page[half] * a.page_stride + (int64_t)slot * a.slot_stride : 0;
            live[half] = __ballot_sync(~0u, ok);
            // keys outside the unit's range are hidden by the rows' limits: only a bad page counts
            shown[half] = __ballot_sync(~0u, ok || key < u.key_lo || key >= u.key_hi);
            page[half] = page_of(j + 1, half);
          }
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            if (kv)
              value_slot(it, j);
            else
              key_slot(it);
            unsigned long long* landed = kv ? &sh.v_landed[it % NV] : &sh.k_landed[it % NS];
            if (kv == 0 && lane == 0) {
              sh.key_ok[it % (2 * NS)][lw * 2] = shown[0];
              sh.key_ok[it % (2 * NS)][lw * 2 + 1] = shown[1];
              mbar_arrive(landed);
            }
            const T* src = kv ? vc : kc;
            const uint32_t dst = kv ? v_smem + it % NV * kTile : k_smem + it % NS * kTile;
            copy_rows(src, off[0], live[0], dst, lw * 64);
            copy_rows(src, off[1], live[1], dst, lw * 64 + 32);
            cp_async_arrive(smem_addr(landed));
          }
        }
        ++seg;
        t += cnt;
        if (t >= span.t1) break;
        unit_begin = t;
        next_unit<kChunkRows, kChunkKeys>(P, &u);
      }
      cp_async_wait_all();
    } else if (lane == 0) {
      // The copies are ordinary writes, the products read by the async proxy: the fence between
      // them costs a hundred cycles or so, which the issuing warp has not got.
      for (int i = 0; i < tiles; ++i) {
        if (!bounded_wait(&sh.k_landed[i % NS], (i / NS) & 1, &sh.limit)) break;
        fence_async_proxy();
        mbar_arrive(&sh.k_full[i % NS]);
        if (!bounded_wait(&sh.v_landed[i % NV], (i / NV) & 1, &sh.limit)) break;
        fence_async_proxy();
        mbar_arrive(&sh.v_full[i % NV]);
      }
    }
  } else {
    // ------------------------------------------------------------------ products
    {
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
        alive = __all_sync(~0u, bounded_wait(bar, parity, &sh.limit)) && alive;
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
            if (kTma) values_ready(it);
            keys_ready(it + 1);  // without TMA handed over after the values of tile it
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
        __syncwarp();
      }
    }
  }
  if (sh.limit.dead) {  // about a millisecond after a wait ran out every copy has landed
    const long long start = clock64();
    for (int i = 0; i < 1 << 16 && clock64() - start < 2000000; ++i) __nanosleep(1000);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 10) tmem_free512(tmem);
  if (tid == 0 && sh.limit.dead) *P.gave_up = 1;
}

}  // namespace clsample
