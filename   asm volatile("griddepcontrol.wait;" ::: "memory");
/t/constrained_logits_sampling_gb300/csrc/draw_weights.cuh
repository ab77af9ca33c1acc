// What the kernels that draw a token from a row of probabilities share: probabilities as integers,
// a row's weights in 16-byte vectors, and their sums over the warps of a cluster's CTAs.
#pragma once

#include "paged.cuh"

namespace clsample {

constexpr int kDrawThreads = 256;
constexpr int kCtasPerSm = 4;
constexpr int kWarps = kDrawThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kLoad = 128;    // vectors that a warp loads at once
constexpr int kBatch = 256;  // vectors of a warp between two marks: at most 32 batches, a thread a vector
constexpr int kMaxVocab = 262144;

// floor(2^40 p) for p in [0, 1], as hi 2^23 + lo, hi = floor(2^17 p) and lo = floor(2^23 times
// the rest).  Adding 2^23 and truncating leaves an integer below 2^23 in a float's low bits;
// the rest is exact.  Four float32 operations, on two numbers at once: a conversion to 64 bits
// would run in the float64 unit, whose rate here bounds a call at four times the memory's time.
constexpr int kIntBits = 0x4b000000;  // of 2^23
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
struct Mass2 {
  int hi[2], lo[2];  // with kIntBits added to each
  __device__ __forceinline__ Mass2(float p0, float p1) {
    const uint64_t p = two(p0, p1), k17 = two(131072.f, 131072.f), k23 = two(8388608.f, 8388608.f);
    const uint64_t minus = two(-1.f, -1.f);
    uint64_t y, rest, z;
    asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(p), "l"(k17), "l"(k23));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(rest) : "l"(y), "l"(minus), "l"(k23));  // -hi
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(rest) : "l"(p), "l"(k17), "l"(rest));
    asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(z) : "l"(rest), "l"(k23), "l"(k23));
    asm("mov.b64 {%0, %1}, %2;" : "=r"(hi[0]), "=r"(hi[1]) : "l"(y));
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo[0]), "=r"(lo[1]) : "l"(z));
  }
};
__device__ __forceinline__ int64_t mass_of(int hi, int lo) { return ((int64_t)hi << 23) + lo; }

__device__ __forceinline__ bool bad_prob(float p) { return !(p >= 0.f && p <= 1.f); }

// Whether any of the probabilities seen was outside [0, 1] or NaN.
struct Range {
  float lo = 0.f, hi = 0.f;
  __device__ __forceinline__ void see(float p, float q) {
    asm("min.f32 %0, %0, %1, %2;" : "+f"(lo) : "f"(p), "f"(q));
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(hi) : "f"(p), "f"(q));  // keeps a NaN
  }
  __device__ __forceinline__ bool bad() const { return !(lo >= 0.f && hi <= 1.f); }
};

__device__ __forceinline__ float load_prob(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_prob(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }

__device__ __forceinline__ void widen16(const uint32_t (&w)[4], float (&x)[4], const float*) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void widen16(const uint32_t (&w)[4], float (&x)[8], const __nv_bfloat16*) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Pair<__nv_bfloat16>::widen(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <class P>
__device__ __forceinline__ int misaligned(const P* row) {  // elements past a 16-byte boundary
  return (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(P));
}

// What is drawn from: the target row, less the draft's row (q) or less everything at one
// token (hole), or neither.  The row is taken in 16-byte vectors that are aligned in p: vector
// v has the tokens v N - a .. v N - a + N - 1, a = misaligned(p), those of them that exist.  q
// may be aligned otherwise: its vector is then put together from the two that hold it.
// kTree: less the draft's row times `taken` (products rounded to float32), or less everything at the
// tokens whose bits are set in `holes` (shared memory, N bits a vector from vector hole_base on).
template <class P, bool kTree = false>
struct Weights {
  static constexpr int N = 16 / sizeof(P);
  const P* p;
  const P* q;
  int hole, V, a, turn;  // turn: elements by which q's vectors lie later than p's
  float taken;
  const uint32_t* holes;
  int hole_base;
  __device__ __forceinline__ void set(const P* p_row, const P* q_row, int hole_at, int vocab) {
    p = p_row;
    q = q_row;
    hole = hole_at;
    V = vocab;
    a = misaligned(p);
    turn = q ? (misaligned(q) - a) & (N - 1) : 0;
  }
  __device__ __forceinline__ int vectors() const { return (V + a + N - 1) / N; }
  // vectors whose loads stay within the rows, in p and in q
  __device__ __forceinline__ int whole_from() const { return (a + turn + N - 1) / N; }
  __device__ __forceinline__ int whole_to() const { return max(0, (V + a - (turn ? N - turn : 0)) / N); }

  // tokens of vector v that have no weight, a bit each
  __device__ __forceinline__ uint32_t hidden(int v) const {
    if constexpr (kTree) {
      if (!holes) return 0;
      const uint32_t at = (uint32_t)(v - hole_base) * N;
      return holes[at >> 5] >> (at & 31) & ((1u << N) - 1);
    } else {
      const int at = hole + a - v * N;  // of the hole in the vector
      return hole >= 0 && at >= 0 && at < N ? 1u << at : 0u;
    }
  }
  __device__ __forceinline__ float less(float y) const { return kTree ? y * taken : y; }

  // 16 bytes of a row from token t0 on, of which the aligned vector before starts `shift` earlier
  __device__ __forceinline__ uint4 bits(const P* row, int t0, int shift) const {
    const uint4* at = reinterpret_cast<const uint4*>(row + t0 - shift);
    const uint4 v = __ldg(at);
    if (shift == 0) return v;
    const uint4 u = __ldg(at + 1);
    uint32_t z[9] = {v.x, v.y, v.z, v.w, u.x, u.y, u.z, u.w, 0};
    const int bytes = shift * (int)sizeof(P);
    if (bytes & 8)
#pragma unroll
      for (int i = 0; i < 7; ++i) z[i] = z[i + 2];
    if (bytes & 4)
#pragma unroll
      for (int i = 0; i < 7; ++i) z[i] = z[i + 1];
    const int b = (bytes & 2) * 8;
    return make_uint4(__funnelshift_r(z[0], z[1], b), __funnelshift_r(z[1], z[2], b), __funnelshift_r(z[2], z[3], b),
                      __funnelshift_r(z[3], z[4], b));
  }
  __device__ __forceinline__ void unpack(uint4 v, float (&x)[N]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    widen16(w, x, p);
  }
  // a vector's tokens one by one, those that there are
  __device__ __forceinline__ void edge(const P* row, int t0, float (&x)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = t0 + i >= 0 && t0 + i < V ? load_prob(row + t0 + i) : 0.f;
  }
  __device__ __forceinline__ void values(int v, float (&x)[N], float (&y)[N]) const {
    const int t0 = v * N - a;
    if (v >= whole_from() && v < whole_to()) {
      unpack(bits(p, t0, 0), x);
      if (q) unpack(bits(q, t0, turn), y);
    } else {
      edge(p, t0, x);
      if (q) edge(q, t0, y);
    }
  }
  // The weights' sum.  Where p > q, P >= Q, and elsewhere P <= Q.
  __device__ __forceinline__ int64_t sum_of(int v, const float (&x)[N], const float (&y)[N], Range* range) const {
    int hi = 0, lo = 0;  // of at most eight weights
    if (q) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        range->see(x[i], y[i]);
        range->see(x[i + 1], y[i + 1]);
        const float z[2] = {less(y[i]), less(y[i + 1])};
        const Mass2 mp(x[i], x[i + 1]), mq(z[0], z[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (x[i + e] > z[e]) {
            hi += mp.hi[e] - mq.hi[e];
            lo += mp.lo[e] - mq.lo[e];
          }
      }
    } else {
      const int t0 = v * N - a;
      const uint32_t gone = kTree ? hidden(v) : 0;
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        range->see(x[i], x[i + 1]);
        const Mass2 mp(x[i], x[i + 1]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (kTree ? !(gone >> (i + e) & 1) : t0 + i + e != hole) {
            hi += mp.hi[e] - kIntBits;
            lo += mp.lo[e] - kIntBits;
          }
      }
    }
    return mass_of(hi, lo);
  }
  __device__ __forceinline__ void vector(int v, int64_t (&w)[N]) const {
    float x[N], y[N];
    values(v, x, y);
    const uint32_t gone = hidden(v);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float z[2] = {q ? less(y[i]) : 0.f, q ? less(y[i + 1]) : 0.f};
      const Mass2 mp(x[i], x[i + 1]), mq(z[0], z[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w[i + e] = (q && x[i + e] <= z[e]) || (gone >> (i + e) & 1)
                       ? 0
                       : mass_of(mp.hi[e] - mq.hi[e], mp.lo[e] - mq.lo[e]);
    }
  }
  // Sum over a warp's vectors first .. end - 1, kLoad at a time with four loads of each row in
  // flight; the lane's sum of each batch is left in marks[batch * kDrawThreads].
  __device__ __forceinline__ int64_t sum_range(int first, int end, Range* range, int64_t* marks) const {
    const int lane = threadIdx.x & 31, from = whole_from(), to = min(end, whole_to());
    int64_t total = 0, sum = 0;
    for (int v0 = first; v0 < end; v0 += kLoad) {  // uniform over the warp
      if (v0 >= from && v0 + kLoad <= to) {
        uint4 x4[4], y4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x4[k] = bits(p, (v0 + 32 * k + lane) * N - a, 0);
        if (q) {
#pragma unroll
          for (int k = 0; k < 4; ++k) y4[k] = bits(q, (v0 + 32 * k + lane) * N - a, turn);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x[N], y[N];
          unpack(x4[k], x);
          unpack(y4[k], y);
          sum += sum_of(v0 + 32 * k + lane, x, y, range);
        }
      } else {
#pragma unroll 1
        for (int v = v0 + lane; v < min(end, v0 + kLoad); v += 32) {
          float x[N], y[N];
          values(v, x, y);
          sum += sum_of(v, x, y, range);
        }
      }
      if (v0 + kLoad >= end || (v0 + kLoad - first) % kBatch == 0) {
        *marks = sum;
        marks += kDrawThreads;
        total += sum;
        sum = 0;
      }
    }
    return total;
  }
};

__device__ __forceinline__ int64_t warp_total(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Shared memory for the marks: a row may take one vector more than its tokens fill.
template <class P, int C>
__host__ __device__ constexpr int marks_words(int V) {
  constexpr int N = 16 / sizeof(P);
  const int vectors = (V + 2 * N - 2) / N, share = (vectors + C - 1) / C, part = (share + kWarps - 1) / kWarps;
  return (part + kBatch - 1) / kBatch * kDrawThreads;
}
template <class P, int C>
int marks_bytes(int V) {
  return marks_words<P, C>(V) * (int)sizeof(int64_t);
}

}  // namespace clsample
