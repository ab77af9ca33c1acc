// The last launch of an attention call: joins the parts of units that span boundaries cut, and
// writes the statuses.
//
// A unit cut into few parts has eight warps on as many rows, one of few rows over a long key
// axis (parts by the hundred) eight warps on the parts of the same rows, which meet in shared
// memory: reading parts is bound by the latency of L2, so each thread has several in flight.
// (Joined by the last CTA of each unit instead, on an earlier version, 50 rows over 130000 keys took
// 152 us against 84.)
// Parts are joined in key order, in an order that depends on the lengths alone.
#pragma once

#include "attn_chunk.cuh"
#include "attn_stream.cuh"

namespace clsample {

constexpr int kJoinThreads = 256;
constexpr int kFewParts = 8;
constexpr int kMaxCuts = 1024;  // CTAs of both kernels

struct JoinParams {
  AttnParams p;        // of the stream kernel's launch
  const float* chunk_partial;
  const CutUnit* chunk_cut;
  int chunk_ctas;      // 0: the chunk kernel was not launched
  int stream_ctas;
};

// Statuses: one CTA per sequence at a time looks at its lengths and at every page id that
// the call touches.
template <int NT, bool kTree>
__device__ __forceinline__ bool attention_bad(const AttnParams& P, int b) {
  const clsample_attention_args_t& a = P.a;
  const Seq s = load_seq(a.cu_new, a.kv_lens, b, a.T, P.capacity, a.max_new);
  int bad = !s.ok || (kTree && s.n > s.len);
  if (kTree && !bad && P.tree.positions)
    for (int i = threadIdx.x; i < s.n; i += NT) {
      const int pos = __ldg(P.tree.positions + s.q0 + i);
      bad |= pos < s.len - s.n || pos >= s.len;
    }
  if (s.ok && s.n > 0 && s.len > 0 && !(kTree && s.n > s.len)) {
    const int lo = a.window > 0 ? max(0, s.len - s.n - a.window + 1) : 0;
#pragma unroll 8
    for (int p = lo / a.page_size + threadIdx.x; p <= (s.len - 1) / a.page_size; p += NT) {
      const int id = __ldg(a.page_table + (int64_t)b * a.table_stride + p);
      bad |= id < 0 || id >= a.num_pages;
    }
  }
  return __syncthreads_or(bad);
}

// NV times four sums of one row, over parts: o and l are relative to m.
template <int NV>
struct RowSum {
  float m, l;
  float4 o[NV];
  __device__ __forceinline__ void clear() {
    m = __int_as_float(0xff800000);
    l = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void add(float mc, float lc, const float4 (&v)[NV]) {
    const float mn = fmaxf(m, mc);
    const float f = m == mn ? 1.f : exp2_fast(m - mn), fc = mc == mn ? 1.f : exp2_fast(mc - mn);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      o[i] = make_float4(o[i].x * f + v[i].x * fc, o[i].y * f + v[i].y * fc, o[i].z * f + v[i].z * fc,
                         o[i].w * f + v[i].w * fc);
    l = l * f + lc * fc;
    m = mn;
  }
};

// Parts first, first + step, .. below `count`; load(part, m, l, v).
template <int NV, class Load>
__device__ __forceinline__ void sum_parts(RowSum<NV>* r, int first, int step, int count, Load load) {
  constexpr int kAhead = NV == 1 ? 8 : 2;
  r->clear();
  for (int p0 = first; p0 < count; p0 += kAhead * step) {
    float m[kAhead], l[kAhead];
    float4 v[kAhead][NV];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (p0 + k * step < count) load(p0 + k * step, &m[k], &l[k], v[k]);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (p0 + k * step < count) r->add(m[k], l[k], v[k]);
  }
}

template <class T, int D, int NV>
__device__ __forceinline__ void finish_row(const AttnParams& P, const CutUnit& u, int r, int d, const RowSum<NV>& s) {
  const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
  const int row = u.row0 + (u.pair ? r & 127 : r), token = u.q0 + token_of(P, row);
  const int head = (u.h + (u.pair ? r >> 7 : 0)) * P.g + head_of(P, row);
  T* dst = (T*)P.a.out + (int64_t)token * P.a.o_stride_t + (int64_t)head * P.a.o_stride_h + d;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    *reinterpret_cast<uint2*>(dst + 4 * i) = make_uint2(Pair<T>::narrow(s.o[i].x * inv, s.o[i].y * inv),
                                                        Pair<T>::narrow(s.o[i].z * inv, s.o[i].w * inv));
  if (d == 0 && P.a.lse) P.a.lse[(int64_t)token * P.a.Hq + head] = lse_of(s.m, s.l);
}

// R: rows of a unit of the stream kernel
template <class T, int D, bool kTree = false, int R = kStreamRows>
__global__ void __launch_bounds__(kJoinThreads, 2) attn_join_kernel(const __grid_constant__ JoinParams J) {
  const AttnParams& P = J.p;
  constexpr int kCols = D / 16;                  // of 16 elements
  constexpr int kChunkStep = 32 * (8 / kCols);   // rows of a chunk unit's block item with few parts
  constexpr int kStreamStep = 8 * (32 / (D / 4));  // rows of a stream unit's
  constexpr int kPerThread = kMaxCuts / kJoinThreads;
  __shared__ int warp_sum[kJoinThreads / 32];
  __shared__ CutUnit cuts[kMaxCuts];
  __shared__ int unit_is, unit_at;
  __shared__ float part_m[8][32], part_l[8][32];
  __shared__ float part_o[8][32][17];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The first status of each CTA rests on the call's inputs alone, and is found while the grids before end.  (Sound
  // as long as the call's first launch has waited for all work before it, which an ordinary launch has.)
  bool bad = false;
  if (P.a.row_status && (int)blockIdx.x < P.a.B) bad = attention_bad<kJoinThreads, kTree>(P, blockIdx.x);
  wait_for_earlier_grids();
  // Thread i has the cut units 4 i .. 4 i + 3, and how many block items they make.
  const int entries = J.chunk_ctas + J.stream_ctas;
  int items[kPerThread], before = 0;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int e = tid * kPerThread + k;
    items[k] = 0;
    if (e < entries) {
      const CutUnit u = e < J.chunk_ctas ? J.chunk_cut[e] : P.cut[e - J.chunk_ctas];
      cuts[e] = u;
      const bool few = u.c1 - u.c0 < kFewParts;
      const int rows = u.pair ? 128 + u.rows : u.rows;  // (a pair's second rows begin at 128)
      if (e < J.chunk_ctas)
        items[k] = few ? (rows + kChunkStep - 1) / kChunkStep : (rows + 31) / 32 * kCols;
      else
        items[k] = few ? (u.rows + kStreamStep - 1) / kStreamStep : u.rows;
    }
    before += items[k];
  }
  const int own = before;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(~0u, before, o);
    if (lane >= o) before += up;
  }
  if (lane == 31) warp_sum[warp] = before;
  __syncthreads();
  before -= own;
  int total = 0;
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) {
    if (i < warp) before += warp_sum[i];
    total += warp_sum[i];
  }

  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    __syncthreads();  // the last item's unit and sums have been read
    int at = item - before;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      if (at >= 0 && at < items[k]) {
        unit_is = tid * kPerThread + k;
        unit_at = at;
      }
      at -= items[k];
    }
    __syncthreads();
    const CutUnit u = cuts[unit_is];
    at = unit_at;
    const int parts = u.c1 - u.c0 + 1;
    const bool few = parts <= kFewParts;
    if (unit_is < J.chunk_ctas) {
      // a slot: four sums of each of 256 rows, the next four of each, ..; one lane a row
      const int r = few ? at * kChunkStep + warp / kCols * 32 + lane : at / kCols * 32 + lane;
      const int d = (few ? warp % kCols : at % kCols) * 16;
      const bool live = u.pair ? r < 256 && (r & 127) < u.rows : r < u.rows;
      auto load = [&](int part, float* m, float* l, float4 (&v)[4]) {
        const float* s = J.chunk_partial + (int64_t)((u.c0 + part) * 2 + (part == 0 ? 1 : 0)) * (kChunkRows * (D + 2));
        *m = __ldcg(s + kChunkRows * D + r);
        *l = __ldcg(s + kChunkRows * D + kChunkRows + r);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __ldcg(reinterpret_cast<const float4*>(s + (d + 4 * i) * kChunkRows + r * 4));
      };
      RowSum<4> sum;
      sum.clear();
      if (live) sum_parts<4>(&sum, few ? 0 : warp, few ? 1 : 8, parts, load);
      if (few) {
        if (live) finish_row<T, D, 4>(P, u, r, d, sum);
        continue;
      }
      part_m[warp][lane] = sum.m;
      part_l[warp][lane] = sum.l;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        part_o[warp][lane][4 * i] = sum.o[i].x;
        part_o[warp][lane][4 * i + 1] = sum.o[i].y;
        part_o[warp][lane][4 * i + 2] = sum.o[i].z;
        part_o[warp][lane][4 * i + 3] = sum.o[i].w;
      }
      __syncthreads();
      if (warp < 4 && live) {  // four sums each
        RowSum<1> all;
        all.clear();
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float* o = &part_o[w][lane][warp * 4];
          const float4 v[1] = {make_float4(o[0], o[1], o[2], o[3])};
          all.add(part_m[w][lane], part_l[w][lane], v);
        }
        finish_row<T, D, 1>(P, u, r, d + warp * 4, all);
      }
    } else {
      // a slot: rows of D sums; D / 4 lanes a row
      constexpr int kPer = D / 4, kRowsPerWarp = 32 / kPer;
      const int sub = lane / kPer, d = lane % kPer * 4;
      const int r = few ? at * kStreamStep + warp * kRowsPerWarp + sub : at;
      const bool live = r < u.rows;
      auto load = [&](int part, float* m, float* l, float4 (&v)[1]) {
        const float* s = P.partial + (int64_t)((u.c0 + part) * 2 + (part == 0 ? 1 : 0)) * (R * (D + 2));
        *m = __ldcg(s + R * D + r);
        *l = __ldcg(s + R * D + R + r);
        v[0] = __ldcg(reinterpret_cast<const float4*>(s + r * D + d));
      };
      RowSum<1> sum;
      sum.clear();
      if (live) sum_parts<1>(&sum, few ? 0 : warp * kRowsPerWarp + sub, few ? 1 : 8 * kRowsPerWarp, parts, load);
      if (few) {
        if (live) finish_row<T, D, 1>(P, u, r, d, sum);
        continue;
      }
      part_m[warp][lane] = sum.m;
      part_l[warp][lane] = sum.l;
      part_o[warp][lane][0] = sum.o[0].x;
      part_o[warp][lane][1] = sum.o[0].y;
      part_o[warp][lane][2] = sum.o[0].z;
      part_o[warp][lane][3] = sum.o[0].w;
      __syncthreads();
      if (tid < kPer) {
        RowSum<1> all;
        all.clear();
#pragma unroll
        for (int w = 0; w < 8 * kRowsPerWarp; ++w) {
          const int wi = w / kRowsPerWarp, li = w % kRowsPerWarp * kPer + tid;
          const float* o = part_o[wi][li];
          const float4 v[1] = {make_float4(o[0], o[1], o[2], o[3])};
          all.add(part_m[wi][li], part_l[wi][li], v);
        }
        finish_row<T, D, 1>(P, u, r, tid * 4, all);
      }
    }
  }
  if (!P.a.row_status) return;
  const bool gave_up = *P.gave_up != 0;
  for (int b = blockIdx.x; b < P.a.B; b += gridDim.x) {
    if (b >= (int)gridDim.x) bad = attention_bad<kJoinThreads, kTree>(P, b);
    if (tid == 0) P.a.row_status[b] = bad ? CLSAMPLE_ROW_INVALID : gave_up ? CLSAMPLE_ROW_OVERFLOW : CLSAMPLE_ROW_OK;
  }
}

}  // namespace clsample
