// What the operators over a paged cache share: the batch's sequences (rows, lengths,
// pages), element conversions and the host's device check.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "clsample.h"

namespace clsample {

// Host: success if the current device is an sm_103 part (`sms`: its SM count, if asked).  What a
// device is does not change, so it is asked for once.
inline int check_device(int* dev_out = nullptr, int* sms = nullptr) {
  constexpr int kDevices = 64, kOther = -1;
  static std::atomic<int> known[kDevices];  // 0: not asked yet; SMs of an sm_103 part; kOther: another
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return CLSAMPLE_ERR_CUDA;
  int count = dev >= 0 && dev < kDevices ? known[dev].load(std::memory_order_relaxed) : 0;
  if (count == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return CLSAMPLE_ERR_CUDA;
    if (major != 10 || minor != 3) count = kOther;
    if (dev >= 0 && dev < kDevices) known[dev].store(count, std::memory_order_relaxed);
  }
  if (count == kOther) return CLSAMPLE_ERR_DEVICE;
  if (sms) *sms = count;
  if (dev_out) *dev_out = dev;
  return CLSAMPLE_SUCCESS;
}

// Host: sets an attribute of kernel fn, which is asked for once a kernel and device.
template <class Kernel>
cudaError_t allow_once(Kernel* fn, cudaFuncAttribute what, int value, std::atomic<uint64_t>* done) {
  int dev = -1;
  const cudaError_t got = cudaGetDevice(&dev);
  if (got != cudaSuccess) return got;
  const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(fn, what, value);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}
template <class Kernel>
cudaError_t allow_smem_once(Kernel* fn, int bytes, std::atomic<uint64_t>* done) {
  return allow_once(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes, done);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The 16-bit types: widening is exact, narrowing rounds to nearest even.
template <class T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 widen(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t narrow(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <> struct Pair<__half> {
  static __device__ __forceinline__ float2 widen(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
  }
  static __device__ __forceinline__ uint32_t narrow(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <class T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// Positions and rows are int32 with room for their sums and differences.
constexpr int kMaxLen = 1 << 30;

// Positions that a page table holds.
__host__ __device__ inline int capacity_of(int max_pages, int page_size) {
  const int64_t c = (int64_t)max_pages * page_size;
  return c < kMaxLen ? (int)c : kMaxLen;
}

// Rows and length of one sequence, as the arrays state them; ok is false when offsets or
// length cannot be (then n is 0 unless the offsets themselves are in order).
struct Seq {
  int q0, n, len;
  bool ok;
};
__device__ __forceinline__ Seq load_seq(const int32_t* cu, const int32_t* lens, int b, int T, int capacity,
                                        int max_new) {
  const int lo = __ldg(cu + b), hi = __ldg(cu + b + 1), len = __ldg(lens + b);
  Seq s{lo, hi - lo, len, true};
  if (lo < 0 || hi < lo || hi > T) return Seq{0, 0, 0, false};
  if (len < 0 || len > capacity || s.n > max_new) {
    s.len = 0;
    s.ok = false;
  }
  return s;
}

}  // namespace clsample
