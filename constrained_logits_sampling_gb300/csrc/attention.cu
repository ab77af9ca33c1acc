// clsample_chunk_attention: attention of each sequence's newest tokens over its paged cache
// (formulas in include/clsample.h).  Host side: argument checks, the handle's scratch and
// the choice of kernels.
#include <new>

#include "attn_chunk.cuh"
#include "attn_join.cuh"
#include "attn_stream.cuh"

struct clsample_attention {
  int dev, sms;
  unsigned char* scratch;
  int stall;              // of AttnParams
  long long wait_cycles;
};

namespace clsample {
namespace {

constexpr int kStreamCtas = 2;  // per SM
constexpr float kMaxScale = 2.0e38f;  // times log2(e) is still finite
// The scratch, per SM: both kernels' slots (two per CTA, of rows of 128 sums, a maximum and a
// sum), their cut units, and one word for all.
constexpr size_t kChunkSlots = 2 * (size_t)kChunkRows * 130 * sizeof(float);
constexpr size_t kStreamSlots = kStreamCtas * 2 * (size_t)kStreamRows * 130 * sizeof(float);
constexpr size_t kCuts = (1 + kStreamCtas) * sizeof(CutUnit);
constexpr size_t kScratch = kChunkSlots + kStreamSlots + kCuts;
// A launch that may start while the one before it ends.
template <class Kernel, class... Args>
cudaError_t launch_after(Kernel fn, int grid, int threads, int smem, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

// A tensor map of 16-bit elements, 128-byte swizzle, zeros out of bounds; false if there is none.
template <int N>
bool make_map(const AttnParams& P, const void* base, const cuuint64_t (&dims)[N], const int64_t (&strides)[N - 1],
              const cuuint32_t (&box)[N], CUtensorMap* map) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<Encode>(fn);
  }();
  if (!encode) return false;
  cuuint64_t bytes[N - 1];
  cuuint32_t ones[N];
  for (int i = 0; i < N; ++i) {
    if (dims[i] == 0) return false;
    // the stride of a dimension of one element is never used, but has to be valid
    if (i > 0) bytes[i - 1] = dims[i] > 1 ? (cuuint64_t)strides[i - 1] * 2 : 16;
    ones[i] = 1;
  }
  return encode(map, P.a.dtype == CLSAMPLE_T_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                N, const_cast<void*>(base), dims, bytes, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The cache as (element, slot, head, page), in boxes of 64 elements of the slots of a page, of a
// tile's keys at most.
bool cache_map(const AttnParams& P, const void* base, CUtensorMap* map) {
  const clsample_attention_args_t& a = P.a;
  const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.page_size, (cuuint64_t)a.Hkv, (cuuint64_t)a.num_pages};
  const int64_t strides[3] = {a.slot_stride, a.head_stride, a.page_stride};
  const cuuint32_t box[4] = {64, (cuuint32_t)(a.page_size < kChunkKeys ? a.page_size : kChunkKeys), 1, 1};
  return make_map(P, base, dims, strides, box, map);
}

// The queries as (element, head, token), in boxes of 64 elements of a row tile: the heads of a key
// head times as many tokens as make 128 rows.
bool query_map(const AttnParams& P, CUtensorMap* map) {
  const clsample_attention_args_t& a = P.a;
  if (P.g > 128 || 128 % P.g != 0) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
  const int64_t strides[2] = {a.q_stride_h, a.q_stride_t};
  const cuuint32_t box[3] = {64, (cuuint32_t)P.g, (cuuint32_t)(128 / P.g)};
  return make_map(P, a.q, dims, strides, box, map);
}

template <class Kernel>
cudaError_t allow_smem(Kernel fn, int bytes) {
  return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <class T, int D>
cudaError_t launch_chunk(AttnParams P, int sms, cudaStream_t st) {
  // Boxes have to start on the eight rows of the swizzle and fill a tile.  2 x 2048 tokens over
  // 14500 to 15600 keys: 557 us with them, 1215 row by row.
  const int page = P.a.page_size;
  CUtensorMap k_map{}, v_map{}, q_map{};
  const bool boxes = page >= 8 && (page % kChunkKeys == 0 || kChunkKeys % page == 0) &&
                     cache_map(P, P.a.k_cache, &k_map) && cache_map(P, P.a.v_cache, &v_map);
  P.q_box = boxes && query_map(P, &q_map);
  const int bytes = ChunkShape<D>::kBytes;
  auto* fn = boxes ? attn_chunk_kernel<T, D, true> : attn_chunk_kernel<T, D, false>;
  const cudaError_t e = allow_smem(fn, bytes);
  if (e != cudaSuccess) return e;
  fn<<<sms, kChunkThreads, bytes, st>>>(P, k_map, v_map, q_map);
  return cudaGetLastError();
}

// first: of the call
template <class T, int D>
cudaError_t launch_stream(const AttnParams& P, int sms, bool first, cudaStream_t st) {
  const int grid = sms * kStreamCtas;
  auto* fn = attn_stream_kernel<T, D>;
  const int bytes = StreamRing<D>::kBytes;
  const cudaError_t e = allow_smem(fn, bytes);
  if (e != cudaSuccess) return e;
  if (!first) return launch_after(fn, grid, kStreamThreads, bytes, st, P);
  fn<<<grid, kStreamThreads, bytes, st>>>(P);
  return cudaGetLastError();
}

template <class T, int D>
cudaError_t launch(const clsample_attention* h, AttnParams P, cudaStream_t st) {
  // no valid sequence has more rows than this; one that breaks the bound has no keys
  const int64_t rows = P.a.max_new * (int64_t)P.g;
  float* const chunk_partial = reinterpret_cast<float*>(h->scratch);
  float* const stream_partial = reinterpret_cast<float*>(h->scratch + h->sms * kChunkSlots);
  CutUnit* const chunk_cut = reinterpret_cast<CutUnit*>(h->scratch + h->sms * (kChunkSlots + kStreamSlots));
  CutUnit* const stream_cut = chunk_cut + h->sms;
  P.gave_up = reinterpret_cast<int*>(stream_cut + h->sms * kStreamCtas);
  // Sequences of up to 16 packed rows go to the stream kernel, longer ones to the chunk
  // kernel.  256 sequences of 16 rows over 2.3 GB of keys and values: 385 us in the one, 441 in
  // the other; of 24 rows, where the one reads keys twice: 707 and 420.
  const bool chunks = rows > kStreamRows;
  // Beside longer sequences, a few short ones are not worth a launch of their own: 19 ragged
  // sequences on 12 key heads take 31 us alone in the chunk kernel and 35 us in both; 240
  // sequences of one token and 16 of 512, on 8 key heads, 708 and 590.
  const bool alone = chunks && (int64_t)P.a.B * P.a.Hkv <= 4 * h->sms;
  cudaError_t e;
  if (chunks) {
    P.min_rows = alone ? 0 : kStreamRows + 1;
    P.max_rows = 0x7fffffff;
    P.partial = chunk_partial;
    P.cut = chunk_cut;
    if ((e = launch_chunk<T, D>(P, h->sms, st)) != cudaSuccess) return e;
  }
  P.min_rows = 0;
  P.max_rows = chunks ? kStreamRows + 1 : 0x7fffffff;
  P.partial = stream_partial;
  P.cut = stream_cut;
  if (!alone && (e = launch_stream<T, D>(P, h->sms, !chunks, st)) != cudaSuccess) return e;
  const JoinParams J{P, chunk_partial, chunk_cut, chunks ? h->sms : 0, alone ? 0 : h->sms * kStreamCtas};
  return launch_after(attn_join_kernel<T, D>, h->sms * 2, kJoinThreads, 0, st, J);
}

}  // namespace
}  // namespace clsample

extern "C" {

int clsample_attention_create(clsample_attention_t** out) {
  using namespace clsample;
  if (!out) return CLSAMPLE_ERR_NULL;
  *out = nullptr;
  int dev = 0, sms = 0;
  const int rc = check_device(&dev, &sms);
  if (rc != CLSAMPLE_SUCCESS) return rc;
  if (sms * (1 + kStreamCtas) > kMaxCuts) return CLSAMPLE_ERR_DEVICE;
  auto* h = new (std::nothrow) clsample_attention{dev, sms, nullptr, 0, kWaitCycles};
  if (!h) return CLSAMPLE_ERR_CUDA;
  const size_t bytes = sms * kScratch + sizeof(int);
  if (cudaMalloc(&h->scratch, bytes) != cudaSuccess || cudaMemset(h->scratch + sms * kScratch, 0, sizeof(int)) != cudaSuccess ||
      cudaDeviceSynchronize() != cudaSuccess) {
    clsample_attention_destroy(h);
    cudaGetLastError();
    return CLSAMPLE_ERR_CUDA;
  }
  *out = h;
  return CLSAMPLE_SUCCESS;
}

void clsample_attention_destroy(clsample_attention_t* h) {
  if (!h) return;
  if (h->scratch) cudaFree(h->scratch);
  delete h;
}

int clsample_debug_attention_stall(clsample_attention_t* h, int32_t barrier, int32_t slot, int64_t wait_cycles) {
  using namespace clsample;
  if (!h) return CLSAMPLE_ERR_NULL;
  if (barrier < 0 || barrier > kStallSums || slot < 0 || slot > 255 || wait_cycles < 1 || wait_cycles > kWaitCycles)
    return CLSAMPLE_ERR_SHAPE;
  h->stall = barrier ? (barrier << 8) + slot : 0;
  h->wait_cycles = barrier ? wait_cycles : kWaitCycles;
  return CLSAMPLE_SUCCESS;
}

int clsample_chunk_attention(clsample_attention_t* h, const clsample_attention_args_t* a, clsample_stream_t stream) {
  using namespace clsample;
  if (!h || !a) return CLSAMPLE_ERR_NULL;
  if (a->B < 0 || a->B > (1 << 24) - 1 || a->T < 0 || a->T > kMaxLen) return CLSAMPLE_ERR_BATCH;
  if (a->dtype != CLSAMPLE_T_BF16 && a->dtype != CLSAMPLE_T_F16) return CLSAMPLE_ERR_DTYPE;
  if (a->Hkv < 1 || a->Hq < a->Hkv || a->Hq > 65536 || a->Hq % a->Hkv != 0 || (a->D != 64 && a->D != 128) ||
      a->num_pages < 0 || a->page_size < 1 || a->max_pages < 0 || a->max_new < 0 || a->window < 0 ||
      !(a->scale > 0.f && a->scale <= kMaxScale) || (int64_t)a->T * (a->Hq / a->Hkv) > 0x7fffffff - 1024)
    return CLSAMPLE_ERR_SHAPE;
  if (a->table_stride < a->max_pages) return CLSAMPLE_ERR_STRIDE;
  if (a->B == 0) return CLSAMPLE_SUCCESS;
  if (!a->cu_new || !a->kv_lens || (!a->page_table && a->max_pages > 0)) return CLSAMPLE_ERR_NULL;
  if (a->T > 0 && (!a->q || !a->out)) return CLSAMPLE_ERR_NULL;
  if (a->num_pages > 0 && a->T > 0 && (!a->k_cache || !a->v_cache)) return CLSAMPLE_ERR_NULL;
  const int64_t strides = a->q_stride_t | a->q_stride_h | a->o_stride_t | a->o_stride_h | a->page_stride |
                          a->slot_stride | a->head_stride;
  if ((strides & 7) || !aligned16(a->q) || !aligned16(a->out) || !aligned16(a->k_cache) || !aligned16(a->v_cache))
    return CLSAMPLE_ERR_ALIGN;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return CLSAMPLE_ERR_CUDA;
  if (dev != h->dev) return CLSAMPLE_ERR_DEVICE;
  AttnParams P{};
  P.a = *a;
  if (P.a.window > kMaxLen) P.a.window = kMaxLen;  // longer than any sequence
  P.g = a->Hq / a->Hkv;
  P.g_shift = (P.g & (P.g - 1)) == 0 ? __builtin_ctz((unsigned)P.g) : -1;
  P.page_shift = (a->page_size & (a->page_size - 1)) == 0 ? __builtin_ctz((unsigned)a->page_size) : -1;
  P.capacity = capacity_of(a->max_pages, a->page_size);
  P.stall = h->stall;
  P.wait_cycles = h->wait_cycles;
  P.scale_log2 = a->scale * 1.44269504088896341f;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a->dtype == CLSAMPLE_T_BF16)
    e = a->D == 128 ? launch<__nv_bfloat16, 128>(h, P, st) : launch<__nv_bfloat16, 64>(h, P, st);
  else
    e = a->D == 128 ? launch<__half, 128>(h, P, st) : launch<__half, 64>(h, P, st);
  return e == cudaSuccess ? CLSAMPLE_SUCCESS : CLSAMPLE_ERR_CUDA;
}

}  // extern "C"
