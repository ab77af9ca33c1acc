// How an attention call is cut into work, shared by its kernels.
//
// A unit is one tile of query rows of one sequence and one key head: the sequence's n
// tokens times the g query heads of the key head are n g packed rows (row r is token r / g,
// head r % g), cut into tiles of R rows.  A unit walks the keys that any of its rows sees in
// tiles of K keys.  All units' key tiles, laid end to end, are cut into equal spans, one per
// CTA, whatever the sequences' lengths: a unit that lies in one span is finished there, one
// that a span boundary cuts leaves partial sums in the handle's scratch, which a last launch
// joins in key order (attn_join.cuh).  Nothing waits for another CTA.
//
// With kTree the rows see the sequence's new tokens by mask instead of by position
// (clsample_tree_attention): every unit of a sequence then has the same keys, and only the tiles
// from the first new token on look at masks.
#pragma once

#include "paged.cuh"

namespace clsample {

// AttnParams.stall: a barrier of the chunk kernel, in bits 8 and up, and which of its slots.
enum Stall {
  kStallUnit = 1, kStallUnitDone, kStallQueries, kStallQueriesDone, kStallKeysLanded, kStallKeys, kStallValuesLanded,
  kStallValues, kStallTileDone, kStallScores, kStallHalfWeights, kStallWeights, kStallSums
};

struct AttnParams {
  clsample_attention_args_t a;
  int g, g_shift;   // query heads per key head; log2, or -1
  int page_shift;   // log2(page_size), or -1
  int capacity;     // positions that the page table holds
  int min_rows;     // this launch takes the sequences with min_rows <= n g < max_rows
  int max_rows;
  int q_box;        // queries may be copied in boxes of 128 rows
  float* partial;   // scratch: two slots per CTA
  struct CutUnit* cut;  // one per CTA: the unit that starts in its span and ends in another's
  int* gave_up;     // set when a bounded wait ran out
  long long wait_cycles;  // that a wait may take
  int stall;        // where a wait of the chunk kernel is in vain, for tests; 0: nowhere
  float scale_log2; // scale * log2(e)
  clsample_tree_mask_t tree;  // with kTree
};

// A packed row's token and its head among those of the key head.
__device__ __forceinline__ int token_of(const AttnParams& P, int row) {
  return P.g_shift >= 0 ? row >> P.g_shift : row / P.g;
}
__device__ __forceinline__ int head_of(const AttnParams& P, int row) { return row - token_of(P, row) * P.g; }

// 64 trees of 24 to 32 tokens over 200 to 4000 keys on 8 key heads, in the chunk kernel, on an earlier version:
// 125 us with 8, 121 with 12, 117 with 18, 120 with 24 (and 197 with spans of equal tiles).
constexpr int kChunkPad = 18, kStreamPad = 3;

struct CutUnit {
  int rows;          // 0: none, and all else is 0 too: the join counts work by `pair` as well
  int row0, q0, h;   // as in Unit
  int c0, c1;        // the CTAs that have its parts: c0 in its second slot, the others in the first
  int pair;          // of two key heads
};

struct Unit {
  int b, h, qt;       // sequence, key head, row tile
  int q0, n, len;     // the sequence's first row, its rows and length
  int row0, rows;     // packed rows of the tile
  int key_lo, key_hi; // keys that any row sees
  int tile0, tiles;   // key tiles, at least one
};

// Bits lo .. hi of a word, of which only 0 .. 31 exist.
__device__ __forceinline__ uint32_t column_bits(int lo, int hi) {
  const uint32_t upto = hi >= 31 ? ~0u : hi < 0 ? 0u : (2u << hi) - 1;
  return lo <= 0 ? upto : lo > 31 ? 0u : upto & (~0u << lo);
}

// kTree: the words of row t, and which of the n new tokens (0 where the sequence has no keys) j0 ..
// j0 + 31 a row sees; j0 may be negative, and tokens that there are not are not seen.
__device__ __forceinline__ const uint32_t* mask_row(const AttnParams& P, int t) {
  return P.tree.mask + (int64_t)t * P.tree.mask_stride;
}
__device__ __forceinline__ uint32_t mask_word(const uint32_t* row, int n, int j0) {
  const int w = j0 >> 5, words = (n + 31) >> 5;  // (w is rounded down)
  const uint32_t lo = (unsigned)w < (unsigned)words ? __ldg(row + w) : 0u;
  const uint32_t hi = (j0 & 31) && (unsigned)(w + 1) < (unsigned)words ? __ldg(row + w + 1) : 0u;
  return __funnelshift_r(lo, hi, j0 & 31) & column_bits(-j0, n - 1 - j0);
}
// The same for 128 tokens from j0 on.
__device__ __forceinline__ uint4 mask_words(const uint32_t* row, int n, int j0) {
  const int w = j0 >> 5, words = (n + 31) >> 5;
  uint32_t x[5];
#pragma unroll
  for (int k = 0; k < 5; ++k) {  // (volatile: loaded here, not where it is first looked at)
    x[k] = 0;
    if ((unsigned)(w + k) < (unsigned)words)
      asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(x[k]) : "l"(row + w + k));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    x[k] = __funnelshift_r(x[k], x[k + 1], j0 & 31) & column_bits(-j0 - 32 * k, n - 1 - j0 - 32 * k);
  return make_uint4(x[0], x[1], x[2], x[3]);
}
// Where row t, the sequence's new token i, stands for the window.
__device__ __forceinline__ int tree_position(const AttnParams& P, int t, int i, int len, int n) {
  return P.tree.positions ? min(max(__ldg(P.tree.positions + t), len - n), len - 1) : len - n + i;
}

// How spans are measured.  A unit is kPad + tiles times its weight long; a tile belongs to the span
// that holds its first position.  With kTree the weights are what tiles cost (of two row tiles 1.5 us, of
// one 1 us); kPad is what a unit costs beside its tiles: its end, and the wait for masks and for the next
// one's first keys.  Sequences of very different lengths would otherwise leave the CTAs with
// many short units far behind.
//
// kPairs: where a key head has one row tile of 128, a unit is two key heads with one row tile each (a
// pair: heads h and h + 1; the last of an odd number is alone).
template <int R, int K, bool kTree = false, bool kPairs = false>
struct UnitMap {
  static constexpr int kRows = R, kKeys = K;
  static constexpr bool kByMask = kTree, kWeighted = kTree && R > 128;  // weighted: the chunk kernel's
  static constexpr int kPad = !kTree ? 0 : kWeighted ? kChunkPad : kStreamPad;
  static constexpr int kMaxWeight = kPairs ? 4 : kWeighted ? 3 : 1;
  static __device__ __forceinline__ bool pairs(const AttnParams& P, int n) {
    return kPairs && P.a.Hkv > 1 && (int64_t)n * P.g <= 128;
  }
  static __device__ __forceinline__ bool is_pair(const AttnParams& P, const Unit& u) {
    return kPairs && pairs(P, u.n) && u.h + 1 < P.a.Hkv;
  }
  static __device__ __forceinline__ int weight(const AttnParams& P, const Unit& u) {
    return !kWeighted ? 1 : u.rows > 128 ? 3 : kPairs && P.a.Hkv > 1 ? 4 : 2;
  }
  // units of one row tile of a sequence with n rows
  static __device__ __forceinline__ int groups(const AttnParams& P, int n) {
    return pairs(P, n) ? (P.a.Hkv + 1) / 2 : P.a.Hkv;
  }
  static __device__ __forceinline__ Seq seq_of(const AttnParams& P, int b) {
    Seq s = load_seq(P.a.cu_new, P.a.kv_lens, b, P.a.T, P.capacity, P.a.max_new);
    const int64_t rows = (int64_t)s.n * P.g;
    if (rows < P.min_rows || rows >= P.max_rows) s.n = 0;  // another launch's
    if (kTree && s.len < s.n) s.len = 0;  // no keys
    return s;
  }
  static __device__ __forceinline__ int row_tiles(const AttnParams& P, const Seq& s) {
    return (int)(((int64_t)s.n * P.g + R - 1) / R);
  }
  // key range and tiles of row tile qt
  static __device__ __forceinline__ void fill(const AttnParams& P, const Seq& s, int qt, Unit* u) {
    u->q0 = s.q0;
    u->n = s.n;
    u->len = s.len;
    u->qt = qt;
    u->row0 = qt * R;
    u->rows = min(R, s.n * P.g - u->row0);
    if constexpr (kTree) {  // a row's window ends at the first new token or later
      u->key_hi = s.len;
      u->key_lo = P.a.window > 0 ? max(0, s.len - s.n - P.a.window + 1) : 0;
      u->tile0 = u->key_lo / K;
      u->tiles = max(1, (u->key_hi + K - 1) / K - u->tile0);
      return;
    }
    const int first = s.len - s.n + token_of(P, u->row0);  // positions of the first and last row
    const int last = s.len - s.n + token_of(P, u->row0 + u->rows - 1);
    u->key_hi = max(0, min(last + 1, s.len));
    u->key_lo = P.a.window > 0 ? min(max(0, first - P.a.window + 1), u->key_hi) : 0;
    u->tile0 = u->key_lo / K;
    u->tiles = max(1, (u->key_hi + K - 1) / K - u->tile0);
  }
  // length of the units of one key head, or of a pair
  static __device__ __forceinline__ int64_t head_tiles(const AttnParams& P, const Seq& s) {
    const int m = row_tiles(P, s);
    int64_t t = 0;
    Unit u;
    for (int qt = 0; qt < m; ++qt) {
      fill(P, s, qt, &u);
      t += u.tiles * weight(P, u) + kPad;
    }
    return t;
  }
};

// Sum of v over the block, and each thread's exclusive prefix; `buf` holds NT / 32 + 1 values.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* buf, int64_t* exclusive) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t run = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(~0u, run, o);
    if (lane >= o) run += up;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = run;
  __syncthreads();
  int64_t base = 0, total = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    if (i < warp) base += buf[i];
    total += buf[i];
  }
  *exclusive = base + run - v;
  return total;
}

// The length of the whole call's units, and where this CTA's span begins: u is the unit that holds
// position t0 = total * cta / ctas, or the next one if no tile of that begins there or later (t0 is then
// the next one's first).  Returns false without work.
struct Span {
  int64_t total, t0, t1;
  int ctas;  // CTAs with work: those with the lower indices
};
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {  // of numbers >= 0; 64-bit division is slow
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int64_t span_begin(int64_t total, int ctas, int c) {
  const int64_t each = quotient(total, ctas);
  return each * c + (uint32_t)((int)(total - each * ctas) * c) / (uint32_t)ctas;
}

// At position t of a span, at unit u: the place in the unit, how many of its tiles are this CTA's, and
// whether the span ends with it.
template <class M>
__device__ __forceinline__ int tiles_before(const AttnParams& P, int64_t at, const Unit& u) {  // that begin before `at`
  if (!M::kWeighted) return (int)min(at, (int64_t)u.tiles);
  const uint32_t x = (uint32_t)min(at, (int64_t)u.tiles * M::kMaxWeight);  // (below 2^26)
  const int w = M::weight(P, u);
  return min(u.tiles, (int)(w == 3 ? (x + 2) / 3 : w == 4 ? (x + 3) / 4 : (x + 1) / 2));
}
template <class M>
__device__ __forceinline__ int tile_in_unit(const AttnParams& P, int64_t t, const Unit& u, int64_t unit_begin) {
  return tiles_before<M>(P, t - unit_begin, u);
}
template <class M>
__device__ __forceinline__ int tiles_here(const AttnParams& P, const Span& span, const Unit& u, int64_t unit_begin,
                                          int64_t t) {
  return tiles_before<M>(P, span.t1 - unit_begin, u) - tile_in_unit<M>(P, t, u, unit_begin);
}
template <class M>
__device__ __forceinline__ bool last_in_span(const AttnParams& P, const Span& span, const Unit& u, int64_t unit_begin) {
  return unit_begin + (int64_t)u.tiles * M::weight(P, u) + M::kPad >= span.t1;
}

template <class M>
__device__ __forceinline__ void next_unit(const AttnParams& P, Unit* u);

template <class M, int NT>
__device__ __forceinline__ bool find_span(const AttnParams& P, Span* span, Unit* u, int64_t* unit_begin) {
  __shared__ int64_t buf[NT / 32 + 1];
  __shared__ Unit found;
  __shared__ int64_t found_begin;
  const int tid = threadIdx.x, B = P.a.B;
  // thread i has the sequences i, i + NT, ..; of up to NT they are read once
  Seq s{0, 0, 0, false};
  int64_t total = 0, ex = 0, per_head = 0;
  for (int base = 0; base < B; base += NT) {
    s.n = 0;
    if (base + tid < B) s = M::seq_of(P, base + tid);
    per_head = M::head_tiles(P, s);
    total += block_scan<NT>(per_head * M::groups(P, s.n), buf, &ex);
  }
  span->total = total;
  // every span holds a tile of the unit that it lies in
  span->ctas = (int)min((int64_t)gridDim.x, M::kByMask ? max((int64_t)1, quotient(total, M::kMaxWeight)) : total);
  if (total == 0) return false;
  if ((int)blockIdx.x >= span->ctas) return false;
  span->t0 = span_begin(total, span->ctas, blockIdx.x);
  span->t1 = span_begin(total, span->ctas, blockIdx.x + 1);
  int64_t seen = 0;
  for (int base = 0; base < B; base += NT) {
    int64_t sum = total;
    if (B > NT) {
      s.n = 0;
      if (base + tid < B) s = M::seq_of(P, base + tid);
      per_head = M::head_tiles(P, s);
      sum = block_scan<NT>(per_head * M::groups(P, s.n), buf, &ex);
    }
    int64_t rest = span->t0 - (seen + ex);
    if (rest >= 0 && rest < per_head * M::groups(P, s.n)) {  // in this thread's sequence
      Unit v;
      v.b = base + tid;
      const int group = (int)quotient(rest, per_head);
      v.h = M::pairs(P, s.n) ? 2 * group : group;
      rest -= group * per_head;
      for (int qt = 0;; ++qt) {
        M::fill(P, s, qt, &v);
        const int64_t length = (int64_t)v.tiles * M::weight(P, v) + M::kPad;
        if (rest < length) break;
        rest -= length;
      }
      found = v;
      found_begin = span->t0 - rest;
    }
    seen += sum;
    if (seen > span->t0) break;  // uniform
  }
  __syncthreads();
  *u = found;
  *unit_begin = found_begin;
  if (M::kPad > 0 && tile_in_unit<M>(P, span->t0, found, found_begin) >= found.tiles) {  // behind the unit's tiles
    *unit_begin += (int64_t)found.tiles * M::weight(P, found) + M::kPad;
    if (*unit_begin >= span->t1) return false;
    next_unit<M>(P, u);
    span->t0 = *unit_begin;
  }
  return true;
}

// On to the next unit; false if the span ends.
template <class M>
__device__ __forceinline__ bool advance(const AttnParams& P, const Span& span, Unit* u, int64_t* unit_begin, int64_t* t) {
  if (last_in_span<M>(P, span, *u, *unit_begin)) return false;
  *unit_begin += (int64_t)u->tiles * M::weight(P, *u) + M::kPad;
  *t = *unit_begin;
  next_unit<M>(P, u);
  return true;
}

// The unit after u (the caller has checked that the span goes on).
template <class M>
__device__ __forceinline__ void next_unit(const AttnParams& P, Unit* u) {
  Seq s{u->q0, u->n, u->len, true};
  if (u->row0 + M::kRows < u->n * P.g) {
    M::fill(P, s, u->qt + 1, u);
    return;
  }
  u->h += M::pairs(P, u->n) ? 2 : 1;
  if (u->h >= P.a.Hkv) {
    u->h = 0;
    do {
      s = M::seq_of(P, ++u->b);
    } while (s.n == 0 && u->b + 1 < P.a.B);
  }
  M::fill(P, s, 0, u);
}

// The CTA whose span holds tile t.
__device__ __forceinline__ int cta_of_tile(const Span& sp, int64_t t) {
  int c = (int)quotient(t * sp.ctas, sp.total);
  while (c + 1 < sp.ctas && span_begin(sp.total, sp.ctas, c + 1) <= t) ++c;
  while (c > 0 && span_begin(sp.total, sp.ctas, c) > t) --c;
  return c;
}

// Called by one thread of each CTA, with the unit that its span ends with: whether the rest of
// it is another's.
template <class M>
__device__ __forceinline__ void note_cut(const AttnParams& P, const Span& span, const Unit& u, int64_t unit_begin) {
  CutUnit c{};
  const int64_t last = unit_begin + (int64_t)(u.tiles - 1) * M::weight(P, u);  // where the last tile is
  if (unit_begin >= span.t0 && last >= span.t1)
    c = CutUnit{u.rows, u.row0, u.q0, u.h, (int)blockIdx.x, cta_of_tile(span, last), M::is_pair(P, u)};
  P.cut[blockIdx.x] = c;
}

// Launches that follow one another without a gap: the next grid may start as this one's blocks
// leave, and takes no result before wait_for_earlier_grids().
__device__ __forceinline__ void let_next_grid_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_earlier_grids() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace clsample
