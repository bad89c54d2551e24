// Attention of one new token per sequence over a window of its last cached positions and its first ones.
#include "paged_attention.cuh"

using namespace adp;

extern "C" int adp_paged_window_attention_workspace(const adp_paged_kv* kv, int32_t n_heads, int32_t window, int32_t sinks,
                                                    uint64_t* bytes) {
  if (window < 1 || sinks < 0) return ADP_ERR_INVALID_ARG;
  return attention_workspace(kv, n_heads, window, sinks, bytes);
}

extern "C" int adp_paged_window_attention(const adp_paged_kv* kv, const void* q, int32_t q_dtype, int32_t n_heads,
                                          int64_t q_stride, float scale, int32_t window, int32_t sinks, void* out,
                                          int64_t out_stride, void* workspace, uint64_t workspace_bytes, int32_t* dev_status,
                                          void* cuda_stream) {
  if (window < 1 || sinks < 0) return ADP_ERR_INVALID_ARG;
  return attention_run<true>(kv, q, q_dtype, n_heads, q_stride, scale, window, sinks, out, out_stride, workspace,
                             workspace_bytes, dev_status, cuda_stream, "adp_paged_window_attention");
}
