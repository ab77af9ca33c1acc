// clsample_tree_attention: attention whose rows see their sequence's new tokens by mask (formulas
// in include/clsample.h).  The kernels are those of clsample_chunk_attention with other limits for
// rows; a source of its own so that the two compile side by side.
#include "attn_launch.cuh"

extern "C" int clsample_tree_attention(clsample_attention_t* h, const clsample_attention_args_t* a,
                                       const clsample_tree_mask_t* tree, clsample_stream_t stream) {
  using namespace clsample;
  if (!tree) return CLSAMPLE_ERR_NULL;
  const int rc = check_attention(h, a);
  if (rc != CLSAMPLE_SUCCESS) return rc;
  if (tree->mask_stride < ((int64_t)a->max_new + 31) / 32) return CLSAMPLE_ERR_STRIDE;
  if (a->B > 0 && a->T > 0 && a->max_new > 0 && !tree->mask) return CLSAMPLE_ERR_NULL;
  return launch_attention<true>(h, a, tree, stream);
}
