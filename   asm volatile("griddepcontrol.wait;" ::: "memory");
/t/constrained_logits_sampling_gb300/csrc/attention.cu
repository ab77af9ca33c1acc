// clsample_chunk_attention: attention of each sequence's newest tokens over its paged cache
// (formulas in include/clsample.h), and the handle that holds the calls' scratch.
#include "attn_launch.cuh"

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
  const int rc = check_attention(h, a);
  return rc == CLSAMPLE_SUCCESS ? launch_attention<false>(h, a, nullptr, stream) : rc;
}

}  // extern "C"
