// Packed K/V rows written into the pages of a cache (16-bit, or e4m3 with one scale per row and head), and
// cached rows read back.
#include <cuda_runtime.h>

#include <type_traits>

#include "../../include/adp.h"
#include "device.cuh"
#include "paged.cuh"

namespace adp {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kTopFast = 3.7057691e-22f;  // 448 x 2^-80: above it no remainder of a quotient that counts underflows

// The sequence that packed row i belongs to: the number of entries of cu[1 .. n] that are at most i (n for
// rows behind the last sequence).  A whole warp asks; 32 entries are compared at a time.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int n, int i, int lane) {
  int lo = 0;
  while (n > 32) {
    const int step = (n + 31) / 32;
    const int at = min((lane + 1) * step, n) - 1;
    const int c = __popc(__ballot_sync(0xFFFFFFFFu, lane * step < n && cu[1 + lo + at] <= i));
    const int skip = min(c * step, n);
    lo += skip;
    n = min(step, n - skip);
  }
  return lo + __popc(__ballot_sync(0xFFFFFFFFu, lane < n && cu[1 + lo + min(lane, max(n - 1, 0))] <= i));
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// x / s correctly rounded, from inv = the correctly rounded 1 / s: one correction of the product (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000", 1990).  A remainder that underflows belongs to a quotient whose
// code is 0 either way.  (An infinity gives NaN.)
__device__ __forceinline__ float divide(float x, float s, float inv) {
  const float y = __fmul_rn(x, inv);
  return fmaf(fmaf(-y, s, x), inv, y);
}

// 8 consecutive elements as they lie in memory.
template <int DT>
struct Raw8 {
  uint32_t w[2 * elem_bytes(DT)];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (DT == DT_E4M3) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int q = 0; q < elem_bytes(DT) / 2; ++q) {
        const uint4 v = *reinterpret_cast<const uint4*>(p + 16 * q);
        w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int q = 0; q < 2 * elem_bytes(DT); ++q) w[q] = 0;
  }
  // The largest magnitude of the LPR lanes' elements (NaN if there is one); 16-bit types two at a time.
  template <int LPR>
  __device__ __forceinline__ float row_max() const {
    if constexpr (DT == DT_F32) {
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(__uint_as_float(w[e])));
#pragma unroll
      for (int d = LPR / 2; d >= 1; d >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      return top;
    } else {
      uint32_t top = w[0] & 0x7FFF7FFFu;
      auto larger = [](uint32_t a, uint32_t b) {
        uint32_t r;
        if constexpr (DT == DT_BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
      };
#pragma unroll
      for (int e = 1; e < 4; ++e) top = larger(top, w[e] & 0x7FFF7FFFu);
#pragma unroll
      for (int d = LPR / 2; d >= 1; d >>= 1) top = larger(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      return max_nan(kv_to_f32((uint16_t)top, DT), kv_to_f32((uint16_t)(top >> 16), DT));
    }
  }
  // In fp32 (exact).
  __device__ __forceinline__ void expand(float (&x)[8]) const {
    if constexpr (DT == DT_F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(w[e]);
    } else {
      load8<DT>(reinterpret_cast<const uint8_t*>(w), x);
    }
  }
};

template <int DT>
__device__ __forceinline__ void store_row8(uint8_t* p, const float (&x)[8]) {
  if constexpr (DT == DT_F32) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 16) = make_float4(x[4], x[5], x[6], x[7]);
  } else if constexpr (DT == DT_E4M3) {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * j], x[4 * j + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * j + 2], x[4 * j + 3]), __NV_SATFINITE, __NV_E4M3);
      w[j] = a | (b << 16);
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack2(x[2 * j], x[2 * j + 1], DT);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Rows into pages (WRITE) or pages into rows, one warp per packed row.  Its K heads and then its V heads are one
// line of 8-element pieces, a piece per lane, so that small rows fill a warp too.  Copying: bound by memory (73,361 bf16
// rows of 8 x 128 read back in 92 us, 6.5 TB/s; 8 pieces in flight per lane instead of 4: the same, and 50 us instead of 47
// for 34,360 rows quantised, 4.5 TB/s).
// Quantising takes a row's absolute maximum over the HD / 8 lanes that hold it (NaN carried along), divides by
// the scale max / 448 and rounds to the nearest code.
template <int ROWDT, int CDT, int HD, bool WRITE>
__global__ void __launch_bounds__(256)
    paged_rows_kernel(PagedView c, uint8_t* rows_k, uint8_t* rows_v, int64_t k_stride, int64_t v_stride,
                      const int32_t* __restrict__ cu, int n_rows, int32_t* status) {
  constexpr int LPR = HD / 8;  // lanes that hold one row of one head
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  // offsets that are wrong are reported, whichever rows they would move
  for (int64_t s = (int64_t)blockIdx.x * 256 + threadIdx.x; s < c.n_seqs; s += (int64_t)gridDim.x * 256)
    if (cu[s + 1] < cu[s] || (s == 0 && cu[0] != 0)) report(status, ADP_ERR_INVALID_ARG);
  if (i >= n_rows) return;
  const int heads = 2 * c.n_kv_heads, piece = (lane % LPR) * 8;
  uint8_t *const rk = rows_k + (int64_t)i * k_stride + piece * elem_bytes(ROWDT);
  uint8_t *const rv = rows_v + (int64_t)i * v_stride + piece * elem_bytes(ROWDT);
  constexpr int kAhead = 4;  // pieces per lane in flight
  constexpr int FROM = WRITE ? ROWDT : CDT;
  Raw8<FROM> raw[kAhead];
  auto row_piece = [&](int hh) {
    const bool is_v = hh >= c.n_kv_heads;
    return (is_v ? rv : rk) + (is_v ? hh - c.n_kv_heads : hh) * (HD * elem_bytes(ROWDT));
  };
  // the packed rows are asked for in front of the look-ups that say where they go
  auto load_rows = [&](int h0) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int hh = h0 + a * (32 / LPR) + lane / LPR;
      if (hh < heads) raw[a].load(row_piece(hh));
      else raw[a].clear();
    }
  };
  if constexpr (WRITE) load_rows(0);
  const int b = find_sequence(cu, c.n_seqs, i, lane);
  int64_t pos = 0;
  int page = -1;
  if (b < c.n_seqs) {
    const int first = cu[b], next = cu[b + 1], len = c.lens[b];
    pos = paged_position(len, next, i);
    if (paged_holds(b, first, next, i))  // else the position may lie behind the sequence's length
      page = paged_page(c.table + (int64_t)b * c.table_width, c.table_width, c.n_pages, c.log2_page, pos);
  } else if (cu[c.n_seqs] <= i) {
    return;  // behind the last sequence
  }
  if (page < 0 && lane == 0) report(status, ADP_ERR_INVALID_ARG);
  if (WRITE && page < 0) return;
  const int slot = (int)(pos & ((1 << c.log2_page) - 1));
  // this lane's piece of head 0 in the page, and the way from head to head (32 bits hold it)
  const int head_step = (HD * elem_bytes(CDT)) << c.log2_page;
  const int64_t cell0 = (int64_t)page * c.page_bytes + ((int64_t)slot * HD + piece) * elem_bytes(CDT);
  uint8_t *const ck = c.k + cell0, *const cv = c.v + cell0;
  const int64_t scale0 = CDT == DT_E4M3 ? (int64_t)page * c.scale_stride + slot : 0;
  for (int h0 = 0; h0 < heads; h0 += kAhead * (32 / LPR)) {
    float sc[kAhead];  // reading e4m3
    if constexpr (WRITE) {
      if (h0 > 0) load_rows(h0);
    } else {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int hh = h0 + a * (32 / LPR) + lane / LPR;
        const bool is_v = hh >= c.n_kv_heads;
        const int h = is_v ? hh - c.n_kv_heads : hh;
        if (hh < heads && page >= 0) {
          raw[a].load((is_v ? cv : ck) + h * head_step);
          if constexpr (CDT == DT_E4M3) sc[a] = (is_v ? c.v_scale : c.k_scale)[scale0 + (h << c.log2_page)];
        } else {
          raw[a].clear();
          sc[a] = 0.0f;
        }
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (h0 + a * (32 / LPR) >= heads) break;
      const int hh = h0 + a * (32 / LPR) + lane / LPR;
      const bool is_v = hh >= c.n_kv_heads, on = hh < heads;
      const int h = is_v ? hh - c.n_kv_heads : hh;
      uint8_t* cell = (is_v ? cv : ck) + h * head_step;
      float* scale = CDT == DT_E4M3 ? (is_v ? c.v_scale : c.k_scale) + scale0 + (h << c.log2_page) : nullptr;
      float x[8];
      raw[a].expand(x);
      if constexpr (CDT == DT_E4M3 && WRITE) {
        const float top = raw[a].template row_max<LPR>();
        float s;
        if (top > kTopFast) {
          s = divide(top, kE4m3Max, 1.0f / kE4m3Max);
        } else {
          s = max_nan(__fdiv_rn(top, kE4m3Max), kScaleMin);
        }
        if (on) {
          if (top > kTopFast) {
            const float inv = __frcp_rn(s);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = divide(x[e], s, inv);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __fdiv_rn(x[e], s);
          }
          store_row8<DT_E4M3>(cell, x);
          if (lane % LPR == 0) *scale = s;
        }
      } else if (on) {
        if constexpr (CDT == DT_E4M3) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(x[e], sc[a]);
        }
        if (WRITE) {
          store_row8<CDT>(cell, x);
        } else {
          store_row8<ROWDT>(row_piece(hh), x);
        }
      }
    }
  }
}

template <bool WRITE>
int paged_rows(const adp_paged_kv* kv, uint8_t* k, uint8_t* v, int32_t rows_dtype, int64_t k_stride, int64_t v_stride,
               const int32_t* cu_rows, int32_t n_rows, int32_t* status, void* stream) {
  PagedView c;
  const int rc = paged_view(kv, &c);
  if (rc) return rc;
  if (rows_dtype != ADP_F16 && rows_dtype != ADP_BF16 && rows_dtype != ADP_F32) return ADP_ERR_UNSUPPORTED_CONFIG;
  if (n_rows < 0 || !cu_rows || ((uintptr_t)cu_rows & 3) || ((uintptr_t)status & 3)) return ADP_ERR_INVALID_ARG;
  if (n_rows == 0 || kv->n_seqs == 0) return ADP_OK;
  const int eb = elem_bytes(rows_dtype);
  const int64_t width = (int64_t)kv->n_kv_heads * kv->head_dim;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return ADP_ERR_INVALID_ARG;
  if (k_stride < width || v_stride < width || (k_stride * eb) % 16 || (v_stride * eb) % 16) return ADP_ERR_INVALID_ARG;
  const int grid = (int)(((int64_t)n_rows + 7) / 8);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto kernel) {
    kernel<<<grid, 256, 0, st>>>(c, k, v, k_stride * eb, v_stride * eb, cu_rows, n_rows, status);
  };
  auto by_rows = [&](auto cdt, auto hd) {
    constexpr int C = decltype(cdt)::value, H = decltype(hd)::value;
    if (rows_dtype == ADP_F16) go(paged_rows_kernel<DT_F16, C, H, WRITE>);
    else if (rows_dtype == ADP_BF16) go(paged_rows_kernel<DT_BF16, C, H, WRITE>);
    else go(paged_rows_kernel<DT_F32, C, H, WRITE>);
  };
  auto by_cache = [&](auto hd) {
    if (kv->dtype == ADP_F16) by_rows(std::integral_constant<int, DT_F16>(), hd);
    else if (kv->dtype == ADP_BF16) by_rows(std::integral_constant<int, DT_BF16>(), hd);
    else by_rows(std::integral_constant<int, DT_E4M3>(), hd);
  };
  if (kv->head_dim == 128) by_cache(std::integral_constant<int, 128>());
  else by_cache(std::integral_constant<int, 64>());
  return cuda_status(cudaGetLastError(), WRITE ? "adp_paged_kv_write" : "adp_paged_kv_read");
}

}  // namespace
}  // namespace adp

using namespace adp;

extern "C" int adp_paged_kv_write(const adp_paged_kv* kv, const void* k, const void* v, int32_t rows_dtype, int64_t k_stride,
                                  int64_t v_stride, const int32_t* cu_rows, int32_t n_rows, int32_t* dev_status,
                                  void* cuda_stream) {
  return paged_rows<true>(kv, static_cast<uint8_t*>(const_cast<void*>(k)), static_cast<uint8_t*>(const_cast<void*>(v)),
                          rows_dtype, k_stride, v_stride, cu_rows, n_rows, dev_status, cuda_stream);
}

extern "C" int adp_paged_kv_read(const adp_paged_kv* kv, void* k, void* v, int32_t rows_dtype, int64_t k_stride,
                                 int64_t v_stride, const int32_t* cu_rows, int32_t n_rows, int32_t* dev_status,
                                 void* cuda_stream) {
  return paged_rows<false>(kv, static_cast<uint8_t*>(k), static_cast<uint8_t*>(v), rows_dtype, k_stride, v_stride, cu_rows,
                           n_rows, dev_status, cuda_stream);
}
