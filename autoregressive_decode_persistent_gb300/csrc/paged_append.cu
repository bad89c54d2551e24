// Packed rows of a fused projection appended to the pages of a cache: queries and keys normed per head (optionally) and
// rotated by their positions, the queries handed back, keys and values put into their pages.
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "../../include/adp.h"
#include "device.cuh"
#include "paged.cuh"
#include "paged_rows.cuh"

namespace adp {
namespace {

struct AppendArgs {
  PagedView c;
  const uint8_t *q, *k, *v;
  uint8_t* out;
  int64_t q_stride, k_stride, v_stride, out_stride;  // bytes
  const int32_t* cu;
  const float *cos, *sin;
  const uint8_t *q_gain, *k_gain;
  int32_t* status;
  int32_t n_rows, n_heads, n_pos, turned;  // turned: pieces of 8 elements that are first of a rotated pair (angles / 8)
  int32_t parts, part_heads;               // warps that share a row, and their heads (of its line of heads)
  int32_t out_dt, gain_dt;
  float eps;
};

// A row's heads are one line: queries, keys, values.  A warp takes one row, or a part of its line where there are few rows;
// its lanes hold pieces of 8 elements, HD / 8 of them a head, kAhead pieces in flight per lane.  Per head: the mean square over
// the head's lanes (a norm's x / sqrt(mean(x^2) + eps) x gain), then the rotation of elements i and i + r by the position's
// angle i (r angles): the partner's piece comes from another lane, and a lane's 8 cosines and sines are the same for all of
// the row's heads.  Everything in fp32, rounded once on the way out (keys to codes x scale in e4m3 pages).
template <int ROWDT, int CDT, int HD>
__global__ void __launch_bounds__(256) paged_append_kernel(const AppendArgs a) {
  constexpr int LPR = HD / 8;  // lanes that hold a head
  constexpr int HPS = 32 / LPR;  // heads of a step of the warp
  constexpr int kAhead = 4;
  constexpr int RB = elem_bytes(ROWDT);
  const PagedView& c = a.c;
  const int lane = threadIdx.x & 31, li = lane % LPR, piece = li * 8;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  // offsets that are wrong are reported, whichever rows they would move
  for (int64_t s = (int64_t)blockIdx.x * 256 + threadIdx.x; s < c.n_seqs; s += (int64_t)gridDim.x * 256)
    if (a.cu[s + 1] < a.cu[s] || (s == 0 && a.cu[0] != 0)) report(a.status, ADP_ERR_INVALID_ARG);
  const int i = (int)(w / a.parts);
  if (i >= a.n_rows) return;
  const int heads = a.n_heads + 2 * c.n_kv_heads;
  const int first = (int)(w % a.parts) * a.part_heads, last = min(first + a.part_heads, heads);
  const uint8_t *const rq = a.q + (int64_t)i * a.q_stride + piece * RB, *const rk = a.k + (int64_t)i * a.k_stride + piece * RB,
                *const rv = a.v + (int64_t)i * a.v_stride + piece * RB;
  Raw8<ROWDT> raw[kAhead];
  // the rows are asked for in front of the look-ups that say where they go
  auto load_rows = [&](int h0) {
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int h = h0 + n * HPS + lane / LPR, hk = h - a.n_heads, hv = hk - c.n_kv_heads;
      if (h < last) raw[n].load(hk < 0 ? rq + h * (HD * RB) : hv < 0 ? rk + hk * (HD * RB) : rv + hv * (HD * RB));
      else raw[n].clear();
    }
  };
  load_rows(first);
  const int b = find_sequence(a.cu, c.n_seqs, i, lane);
  int64_t pos = 0;
  int page = -1;
  if (b < c.n_seqs) {
    const int begin = a.cu[b], next = a.cu[b + 1], len = c.lens[b];
    pos = paged_position(len, next, i);
    if (paged_holds(b, begin, next, i))
      page = paged_page(c.table + (int64_t)b * c.table_width, c.table_width, c.n_pages, c.log2_page, pos);
  } else if (a.cu[c.n_seqs] <= i) {
    return;  // behind the last sequence
  }
  if (page < 0 && lane == 0) report(a.status, ADP_ERR_INVALID_ARG);
  if (page >= 0 && pos >= a.n_pos) {  // no angles
    if (lane == 0) report(a.status, ADP_ERR_CONTEXT_OVERFLOW);
    page = -1;
  }
  const bool there = page >= 0;
  // this lane's angles, and the lane with the other halves of its pairs
  const bool low = li < a.turned, turned = li < 2 * a.turned;
  const int partner = low ? lane + a.turned : turned ? lane - a.turned : lane;
  float cs[8], sn[8];
  if (turned && there) {
    const int64_t at = pos * (a.turned * 8) + (low ? li : li - a.turned) * 8;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(a.cos + at + e)), y = __ldg(reinterpret_cast<const float4*>(a.sin + at + e));
      cs[e] = x.x, cs[e + 1] = x.y, cs[e + 2] = x.z, cs[e + 3] = x.w;
      sn[e] = y.x, sn[e + 1] = y.y, sn[e + 2] = y.z, sn[e + 3] = y.w;
    }
    if (low)
#pragma unroll
      for (int e = 0; e < 8; ++e) sn[e] = -sn[e];
  }
  const int slot = (int)(pos & ((1 << c.log2_page) - 1));
  const int head_step = (HD * elem_bytes(CDT)) << c.log2_page;  // (32 bits hold it, as in the other rows' kernels)
  const int64_t cell0 = (int64_t)page * c.page_bytes + ((int64_t)slot * HD + piece) * elem_bytes(CDT);
  const int64_t scale0 = CDT == DT_E4M3 ? (int64_t)page * c.scale_stride + slot : 0;
  uint8_t* const ro = a.out + (int64_t)i * a.out_stride + piece * elem_bytes(a.out_dt);
#pragma unroll 1
  for (int h0 = first; h0 < last; h0 += kAhead * HPS) {
    if (h0 > first) load_rows(h0);
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      if (h0 + n * HPS >= last) break;
      const int h = h0 + n * HPS + lane / LPR, hk = h - a.n_heads, hv = hk - c.n_kv_heads;
      const bool on = h < last, is_q = hk < 0, is_v = hv >= 0;
      float x[8];
      raw[n].expand(x);
      if (!__all_sync(0xFFFFFFFFu, is_v)) {
        const uint8_t* gain = is_q ? a.q_gain : is_v ? nullptr : a.k_gain;
        if (a.q_gain || a.k_gain) {
          float sum = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
          for (int d = LPR / 2; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
          if (gain) {
            const float f = rsqrtf(sum * (1.0f / HD) + a.eps);
            float g[8];
            if (a.gain_dt == DT_F32) {
              const float4 u = __ldg(reinterpret_cast<const float4*>(gain) + 2 * li), v = __ldg(reinterpret_cast<const float4*>(gain) + 2 * li + 1);
              g[0] = u.x, g[1] = u.y, g[2] = u.z, g[3] = u.w, g[4] = v.x, g[5] = v.y, g[6] = v.z, g[7] = v.w;
            } else if (a.gain_dt == DT_BF16) {
              load8<DT_BF16>(gain + piece * 2, g);
            } else {
              load8<DT_F16>(gain + piece * 2, g);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * f * g[e];
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = __shfl_sync(0xFFFFFFFFu, x[e], partner);
          if (turned && !is_v) x[e] = fmaf(x[e], cs[e], y * sn[e]);
        }
      }
      float top = 0.0f;
      if constexpr (CDT == DT_E4M3) {
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(x[e]));
#pragma unroll
        for (int d = LPR / 2; d >= 1; d >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      }
      if (!on) continue;
      if (is_q) {
        if (!there) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = 0.0f;
        }
        uint8_t* p = ro + h * HD * elem_bytes(a.out_dt);
        if (a.out_dt == DT_BF16) store_row8<DT_BF16>(p, x);
        else if (a.out_dt == DT_F16) store_row8<DT_F16>(p, x);
        else store_row8<DT_F32>(p, x);
      } else if (there) {
        const int hc = is_v ? hv : hk;
        uint8_t* cell = (is_v ? c.v : c.k) + cell0 + hc * head_step;
        if constexpr (CDT == DT_E4M3) {
          const float s = quantise8(x, top);
          if (li == 0) (is_v ? c.v_scale : c.k_scale)[scale0 + ((int64_t)hc << c.log2_page)] = s;
        }
        store_row8<CDT>(cell, x);
      }
    }
  }
}

// Warps that share a row: a row's line of heads is cut while there are fewer rows than warps that the GPU holds.
constexpr int kWarpsPerSm = 24;

}  // namespace
}  // namespace adp

using namespace adp;

extern "C" int adp_paged_kv_append(const adp_paged_kv* kv, const adp_rope* rope, const void* q, const void* k, const void* v,
                                   int32_t rows_dtype, int32_t n_heads, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                   const int32_t* cu_rows, int32_t n_rows, void* out, int32_t out_dtype, int64_t out_stride,
                                   int32_t* dev_status, void* cuda_stream) {
  AppendArgs a{};
  int rc = paged_view(kv, &a.c);
  if (rc) return rc;
  if (!rope) return ADP_ERR_INVALID_ARG;
  auto known = [](int32_t dt) { return dt == ADP_F16 || dt == ADP_BF16 || dt == ADP_F32; };
  if (!known(rows_dtype) || n_heads > 4096) return ADP_ERR_UNSUPPORTED_CONFIG;
  if (n_heads < 0 || n_rows < 0 || !cu_rows || ((uintptr_t)cu_rows & 3) || ((uintptr_t)dev_status & 3)) return ADP_ERR_INVALID_ARG;
  if (n_heads > 0 && !known(out_dtype)) return ADP_ERR_UNSUPPORTED_CONFIG;
  if (rope->n_positions < 0 || rope->rotated < 0 || !(rope->eps >= 0.0f) || !isfinite(rope->eps)) return ADP_ERR_INVALID_ARG;
  if (rope->rotated % 16 || rope->rotated < 16 || rope->rotated > kv->head_dim) return ADP_ERR_UNSUPPORTED_CONFIG;
  if (!rope->cos || !rope->sin || !aligned16(rope->cos) || !aligned16(rope->sin)) return ADP_ERR_INVALID_ARG;
  if (rope->q_gain || rope->k_gain) {
    if (!known(rope->gain_dtype)) return ADP_ERR_UNSUPPORTED_CONFIG;
    if (!aligned16(rope->q_gain) || !aligned16(rope->k_gain)) return ADP_ERR_INVALID_ARG;
  }
  if (n_rows == 0 || kv->n_seqs == 0) return ADP_OK;
  const int eb = elem_bytes(rows_dtype);
  const int64_t width = (int64_t)kv->n_kv_heads * kv->head_dim, q_width = (int64_t)n_heads * kv->head_dim;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return ADP_ERR_INVALID_ARG;
  if (k_stride < width || v_stride < width || (k_stride * eb) % 16 || (v_stride * eb) % 16) return ADP_ERR_INVALID_ARG;
  if (n_heads > 0) {
    if (!q || !out || !aligned16(q) || !aligned16(out) || q_stride < q_width || out_stride < q_width) return ADP_ERR_INVALID_ARG;
    if ((q_stride * eb) % 16 || (out_stride * elem_bytes(out_dtype)) % 16) return ADP_ERR_INVALID_ARG;
  }
  int sms = 0;
  if ((rc = sm_count(&sms))) return rc;
  a.q = static_cast<const uint8_t*>(q);
  a.k = static_cast<const uint8_t*>(k);
  a.v = static_cast<const uint8_t*>(v);
  a.out = static_cast<uint8_t*>(out);
  a.q_stride = q_stride * eb;
  a.k_stride = k_stride * eb;
  a.v_stride = v_stride * eb;
  a.out_stride = n_heads > 0 ? out_stride * elem_bytes(out_dtype) : 0;
  a.cu = cu_rows;
  a.cos = rope->cos;
  a.sin = rope->sin;
  a.q_gain = static_cast<const uint8_t*>(rope->q_gain);
  a.k_gain = static_cast<const uint8_t*>(rope->k_gain);
  a.status = dev_status;
  a.n_rows = n_rows;
  a.n_heads = n_heads;
  a.n_pos = rope->n_positions;
  a.turned = rope->rotated / 16;
  a.out_dt = n_heads > 0 ? out_dtype : ADP_F16;
  a.gain_dt = rope->gain_dtype;
  a.eps = rope->eps;
  const int heads = n_heads + 2 * kv->n_kv_heads, step = 32 / (kv->head_dim / 8);
  const int most = (heads + step - 1) / step, want = sms * kWarpsPerSm / n_rows;
  a.parts = want < 1 ? 1 : want > most ? most : want;
  a.part_heads = (most + a.parts - 1) / a.parts * step;
  a.parts = (heads + a.part_heads - 1) / a.part_heads;
  const int64_t grid = ((int64_t)n_rows * a.parts + 7) / 8;
  if (grid > 0x7FFFFFFF) return ADP_ERR_UNSUPPORTED_CONFIG;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  auto by_rows = [&](auto cdt, auto hd) {
    constexpr int C = decltype(cdt)::value, H = decltype(hd)::value;
    if (rows_dtype == ADP_F16) paged_append_kernel<DT_F16, C, H><<<(unsigned)grid, 256, 0, st>>>(a);
    else if (rows_dtype == ADP_BF16) paged_append_kernel<DT_BF16, C, H><<<(unsigned)grid, 256, 0, st>>>(a);
    else paged_append_kernel<DT_F32, C, H><<<(unsigned)grid, 256, 0, st>>>(a);
  };
  auto by_cache = [&](auto hd) {
    if (kv->dtype == ADP_F16) by_rows(std::integral_constant<int, DT_F16>(), hd);
    else if (kv->dtype == ADP_BF16) by_rows(std::integral_constant<int, DT_BF16>(), hd);
    else by_rows(std::integral_constant<int, DT_E4M3>(), hd);
  };
  if (kv->head_dim == 128) by_cache(std::integral_constant<int, 128>());
  else by_cache(std::integral_constant<int, 64>());
  return cuda_status(cudaGetLastError(), "adp_paged_kv_append");
}
