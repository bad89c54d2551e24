// What the kernels of the paged operators and their host code share.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/adp.h"
#include "device.cuh"
#include "paged.h"
#include "scratch.h"

namespace adp {

constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126, the least scale of an e4m3 row: one of zeros divides by it

__host__ __device__ constexpr int elem_bytes(int dt) { return dt == DT_F32 ? 4 : dt == DT_E4M3 ? 1 : 2; }

// What the kernels take of an adp_paged_kv.
struct PagedView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t page_bytes;    // bytes from one page to the next
  int64_t scale_stride;  // floats from one page's scales to the next's
  const int32_t* table;
  const int32_t* lens;
  int32_t table_width, n_pages, log2_page, n_kv_heads, n_seqs;
};

__device__ __forceinline__ void report(int32_t* status, int32_t code) {
  if (status) *reinterpret_cast<volatile int32_t*>(status) = code;
}

// Two values rounded to nearest even, low | high << 16.
__device__ __forceinline__ uint32_t pack2(float lo, float hi, int dt) {
  if (dt == DT_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

inline int cuda_status(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return ADP_OK;
  char msg[256];
  snprintf(msg, sizeof(msg), "%s: %s", where, cudaGetErrorString(e));
  set_last_error(msg);
  return ADP_ERR_CUDA;
}

// A finite scale for scores in base-2 exponents, kept finite: scores of 0 are 0 under the largest, too.
inline float log2_scale(float scale) {
  const float s = scale * 1.4426950408889634f;
  return s > 3.40282347e38f ? 3.40282347e38f : s < -3.40282347e38f ? -3.40282347e38f : s;
}

// Checks of a cache's description that need no device, and the kernels' view of it.
inline int paged_view(const adp_paged_kv* c, PagedView* out) {
  if (!c || !c->k || !c->v || (c->n_seqs > 0 && (!c->table || !c->lens))) return ADP_ERR_INVALID_ARG;
  if (c->n_seqs < 0 || c->n_pages < 1 || c->table_width < 1 || c->n_kv_heads < 1 || c->page_size < 1)
    return ADP_ERR_INVALID_ARG;
  if (c->dtype != ADP_F16 && c->dtype != ADP_BF16 && c->dtype != ADP_E4M3) return ADP_ERR_UNSUPPORTED_CONFIG;
  if (c->head_dim != 64 && c->head_dim != 128) return ADP_ERR_UNSUPPORTED_CONFIG;
  if (c->page_size > kPagedMaxPage || (c->page_size & (c->page_size - 1))) return ADP_ERR_UNSUPPORTED_CONFIG;
  if (c->n_kv_heads > 1024) return ADP_ERR_UNSUPPORTED_CONFIG;
  int lg = 0;
  while ((1 << lg) < c->page_size) ++lg;
  if (((int64_t)c->table_width << lg) > 0x7FFFFFFFll - 1024) return ADP_ERR_UNSUPPORTED_CONFIG;
  const int eb = elem_bytes(c->dtype);
  const int64_t cells = (int64_t)c->n_kv_heads * c->page_size;
  if (c->page_stride < cells * c->head_dim || (c->page_stride * eb) % 16) return ADP_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v)) return ADP_ERR_INVALID_ARG;
  if (c->dtype == ADP_E4M3) {
    if (!c->k_scale || !c->v_scale || c->scale_stride < cells) return ADP_ERR_INVALID_ARG;
    if (((uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 3) return ADP_ERR_INVALID_ARG;
  }
  if (((uintptr_t)c->table | (uintptr_t)c->lens) & 3) return ADP_ERR_INVALID_ARG;
  *out = PagedView{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->k_scale, c->v_scale, c->page_stride * eb,
                   c->scale_stride, c->table, c->lens, c->table_width, c->n_pages, lg, c->n_kv_heads, c->n_seqs};
  return ADP_OK;
}

// SMs of the current device.
inline int sm_count(int* sms) {
  static int known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e, "cudaGetDevice");
  if (dev < 64 && known[dev]) {
    *sms = known[dev];
    return ADP_OK;
  }
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_status(e, "cudaDeviceGetAttribute");
  if (dev < 64) known[dev] = *sms;
  return ADP_OK;
}

// The shared-memory limit of one kernel (KEY: a type of its own for each), set once per device; a lost race sets
// it twice.
template <class KEY>
cudaError_t allow_smem(const void* kernel, size_t bytes) {
  static bool done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev])) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) done[dev] = true;
  return e;
}

}  // namespace adp
