// Packed rows in pieces of 8 elements: the sequence of a row, pieces as they lie in memory, quantisation to e4m3.  What
// the kernels that write rows into pages have in common.
#pragma once
#include <cuda_runtime.h>

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

// Scale and codes of a row of one head whose largest magnitude is top (NaN where the row holds one): x becomes what
// store_row8<DT_E4M3> rounds to codes.
__device__ __forceinline__ float quantise8(float (&x)[8], float top) {
  float s;
  if (top > kTopFast) {
    s = divide(top, kE4m3Max, 1.0f / kE4m3Max);
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = divide(x[e], s, inv);
  } else {
    s = max_nan(__fdiv_rn(top, kE4m3Max), kScaleMin);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __fdiv_rn(x[e], s);
  }
  return s;
}

// The same for two pieces of a row, as pairs of elements; the scale and its reciprocal are computed once.
__device__ __forceinline__ float quantise16(float2 (&x)[2][4], float top) {
  float s;
  if (top > kTopFast) {
    s = divide(top, kE4m3Max, 1.0f / kE4m3Max);
    const float inv = __frcp_rn(s);
    const float2 inv2 = make_float2(inv, inv), ns2 = make_float2(-s, -s);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // (divide(), two at a time)
        const float2 y = __fmul2_rn(x[k][e], inv2);
        x[k][e] = __ffma2_rn(__ffma2_rn(y, ns2, x[k][e]), inv2, y);
      }
  } else {
    s = max_nan(__fdiv_rn(top, kE4m3Max), kScaleMin);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[k][e] = make_float2(__fdiv_rn(x[k][e].x, s), __fdiv_rn(x[k][e].y, s));
  }
  return s;
}

}  // namespace
}  // namespace adp
