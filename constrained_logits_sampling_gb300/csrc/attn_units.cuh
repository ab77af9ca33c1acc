// How an attention call is cut into work, shared by its kernels.
//
// A unit is one tile of query rows of one sequence and one key head: the sequence's n
// tokens times the g query heads of the key head are n g packed rows (row r is token r / g,
// head r % g), cut into tiles of R rows.  A unit walks the keys that any of its rows sees in
// tiles of K keys.  All units' key tiles, laid end to end, are cut into equal spans, one per
// CTA, whatever the sequences' lengths: a unit that lies in one span is finished there, one
// that a span boundary cuts leaves partial sums in the handle's scratch, which a last launch
// joins in key order (attn_join.cuh).  Nothing waits for another CTA.
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
};

// A packed row's token and its head among those of the key head.
__device__ __forceinline__ int token_of(const AttnParams& P, int row) {
  return P.g_shift >= 0 ? row >> P.g_shift : row / P.g;
}
__device__ __forceinline__ int head_of(const AttnParams& P, int row) { return row - token_of(P, row) * P.g; }

struct CutUnit {
  int rows;          // 0: none
  int row0, q0, h;   // as in Unit
  int c0, c1;        // the CTAs that have its parts: c0 in its second slot, the others in the first
};

struct Unit {
  int b, h, qt;       // sequence, key head, row tile
  int q0, n, len;     // the sequence's first row, its rows and length
  int row0, rows;     // packed rows of the tile
  int key_lo, key_hi; // keys that any row sees
  int tile0, tiles;   // key tiles, at least one
};

template <int R, int K>
struct UnitMap {
  static __device__ __forceinline__ Seq seq_of(const AttnParams& P, int b) {
    Seq s = load_seq(P.a.cu_new, P.a.kv_lens, b, P.a.T, P.capacity, P.a.max_new);
    const int64_t rows = (int64_t)s.n * P.g;
    if (rows < P.min_rows || rows >= P.max_rows) s.n = 0;  // another launch's
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
    const int first = s.len - s.n + token_of(P, u->row0);  // positions of the first and last row
    const int last = s.len - s.n + token_of(P, u->row0 + u->rows - 1);
    u->key_hi = max(0, min(last + 1, s.len));
    u->key_lo = P.a.window > 0 ? min(max(0, first - P.a.window + 1), u->key_hi) : 0;
    u->tile0 = u->key_lo / K;
    u->tiles = max(1, (u->key_hi + K - 1) / K - u->tile0);
  }
  // key tiles of one key head of a sequence
  static __device__ __forceinline__ int64_t head_tiles(const AttnParams& P, const Seq& s) {
    const int m = row_tiles(P, s);
    int64_t t = 0;
    Unit u;
    for (int qt = 0; qt < m; ++qt) {
      fill(P, s, qt, &u);
      t += u.tiles;
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

// The whole call's key tiles, and where this CTA's span begins: u is the unit that holds
// tile t0 = total * cta / ctas, *offset the tile's place in it.  Returns false without work.
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

template <int R, int K, int NT>
__device__ __forceinline__ bool find_span(const AttnParams& P, Span* span, Unit* u, int64_t* unit_begin) {
  using M = UnitMap<R, K>;
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
    total += block_scan<NT>(per_head * P.a.Hkv, buf, &ex);
  }
  span->total = total;
  span->ctas = (int)min((int64_t)gridDim.x, total);
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
      sum = block_scan<NT>(per_head * P.a.Hkv, buf, &ex);
    }
    int64_t rest = span->t0 - (seen + ex);
    if (rest >= 0 && rest < per_head * P.a.Hkv) {  // in this thread's sequence
      Unit v;
      v.b = base + tid;
      v.h = (int)quotient(rest, per_head);
      rest -= v.h * per_head;
      for (int qt = 0;; ++qt) {
        M::fill(P, s, qt, &v);
        if (rest < v.tiles) break;
        rest -= v.tiles;
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
  return true;
}

// The unit after u (the caller has checked that the span goes on).
template <int R, int K>
__device__ __forceinline__ void next_unit(const AttnParams& P, Unit* u) {
  using M = UnitMap<R, K>;
  Seq s{u->q0, u->n, u->len, true};
  if (u->row0 + R < u->n * P.g) {
    M::fill(P, s, u->qt + 1, u);
    return;
  }
  if (++u->h >= P.a.Hkv) {
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
__device__ __forceinline__ void note_cut(const AttnParams& P, const Span& span, const Unit& u, int64_t unit_begin) {
  CutUnit c{0, 0, 0, 0, 0, 0};
  if (unit_begin >= span.t0 && unit_begin + u.tiles > span.t1)
    c = CutUnit{u.rows, u.row0, u.q0, u.h, (int)blockIdx.x, cta_of_tile(span, unit_begin + u.tiles - 1)};
  P.cut[blockIdx.x] = c;
}

// Launches that follow one another without a gap: the next grid may start as this one's blocks
// leave, and takes no result before wait_for_earlier_grids().
__device__ __forceinline__ void let_next_grid_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_earlier_grids() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace clsample
