// Attention of one new token per sequence over all of its cached positions.
#include "paged_attention.cuh"

using namespace adp;

extern "C" int adp_paged_attention_workspace(const adp_paged_kv* kv, int32_t n_heads, uint64_t* bytes) {
  return attention_workspace(kv, n_heads, 0, 0, bytes);
}

extern "C" int adp_paged_attention(const adp_paged_kv* kv, const void* q, int32_t q_dtype, int32_t n_heads, int64_t q_stride,
                                   float scale, void* out, int64_t out_stride, void* workspace, uint64_t workspace_bytes,
                                   int32_t* dev_status, void* cuda_stream) {
  return attention_run<false>(kv, q, q_dtype, n_heads, q_stride, scale, 0, 0, out, out_stride, workspace, workspace_bytes,
                              dev_status, cuda_stream, "adp_paged_attention");
}
