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

constexpr int kAppendThreads = 32;  // a warp: the last CTAs of a call leave few SMs idle (64: 140 us instead of 137, 256: 148)

constexpr float kLeastMean = 8.0779357e-28f;  // 2^-90: above it no square that counts underflows

// The power of two that brings the larger of a head's largest magnitude and the root of eps to between 1 and 4, as far as fp32 has one.
__device__ __forceinline__ float power_near(float top, float eps) {
  const int of_top = (int)(__float_as_uint(top) >> 23) - 127;
  const int of_eps = eps > 0.0f ? ((int)(__float_as_uint(eps) >> 23) - 127) >> 1 : -126;
  return __uint_as_float((uint32_t)(127 - min(max(max(of_top, of_eps), -126), 126)) << 23);
}

struct AppendArgs {
  PagedView c;
  const uint8_t *q, *k, *v;
  uint8_t* out;
  int64_t q_stride, k_stride, v_stride, out_stride;  // bytes
  const int32_t* cu;
  const float *cos, *sin;
  const uint8_t *q_gain, *k_gain;
  int32_t* status;
  int32_t n_rows, n_heads, n_pos, turned;  // turned: pieces of 8 elements that are the first of rotated pairs
  int32_t parts, part_heads;               // warps that share a row, and their heads (of its line of heads)
  int32_t out_dt, gain_dt;
  float eps;
};

// A row's heads are one line: queries, keys, values.  A warp takes one row, or a part of its line where there are few rows.
// HD / 16 lanes hold a head, two pieces of 8 elements each: a lane with rotated elements has both halves of its pairs (pieces
// u and u + turned), so that the rotation needs no other lane, and the mean square and the largest magnitude take three
// exchanges a head.  A lane's 8 cosines and sines are the same for all of the row's heads.  Per head: a norm's x / sqrt(mean(x^2) +
// eps) x gain (a head whose squares leave fp32's range is scaled first), then x_i cos - x_(i+r) sin and x_(i+r) cos + x_i sin;
// everything in fp32, in pairs where there are instructions for them, and rounded once on the way out (keys to codes x scale
// in e4m3 pages).
// Bound by the bytes where rows are many (34,360 rows of 32 + 16 heads x 128 in bf16: 845 MB in 137 us, 92% of the copy rate), and by
// the look-ups of a row in a line (offsets, length, page, angles) with 16 warps an SM where they are fewer (5,593 rows, normed, to
// e4m3 pages: 127 MB in 37 us, 51%; in thirds of a row 37, in sixths 44).
template <int ROWDT, int CDT, int HD>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const AppendArgs a) {
  constexpr int LPH = HD / 16;    // lanes that hold a head
  constexpr int HPS = 32 / LPH;   // heads of a step of the warp
  constexpr int kAhead = ROWDT == DT_F32 ? 2 : 4;  // steps in flight
  constexpr int RB = elem_bytes(ROWDT);
  const PagedView& c = a.c;
  const int lane = threadIdx.x & 31, u = lane % LPH;
  const int pa = u < a.turned ? u : 2 * u, pb = u < a.turned ? u + a.turned : 2 * u + 1;  // this lane's pieces of a head
  const int64_t w = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  // offsets that are wrong are reported, whichever rows they would move
  for (int64_t s = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x; s < c.n_seqs; s += (int64_t)gridDim.x * kAppendThreads)
    if (a.cu[s + 1] < a.cu[s] || (s == 0 && a.cu[0] != 0)) report(a.status, ADP_ERR_INVALID_ARG);
  const int i = a.parts == 1 ? (int)w : (int)(w / a.parts);
  if (i >= a.n_rows) return;
  const int heads = a.n_heads + 2 * c.n_kv_heads;
  const int first = a.parts == 1 ? 0 : (int)(w - (int64_t)i * a.parts) * a.part_heads, last = min(first + a.part_heads, heads);
  const uint8_t *const rq = a.q + (int64_t)i * a.q_stride, *const rk = a.k + (int64_t)i * a.k_stride,
                *const rv = a.v + (int64_t)i * a.v_stride;
  Raw8<ROWDT> raw[kAhead][2];
  // the rows are asked for in front of the look-ups that say where they go
  auto load_rows = [&](int h0) {
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int h = h0 + n * HPS + lane / LPH, hk = h - a.n_heads, hv = hk - c.n_kv_heads;
      if (h < last) {
        const uint8_t* p = hk < 0 ? rq + h * (HD * RB) : hv < 0 ? rk + hk * (HD * RB) : rv + hv * (HD * RB);
        raw[n][0].load(p + pa * (8 * RB));
        raw[n][1].load(p + pb * (8 * RB));
      } else {
        raw[n][0].clear();
        raw[n][1].clear();
      }
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
  uint8_t* const ro = a.out + (int64_t)i * a.out_stride;
  if (page < 0) {  // its queries become zeros
    const int row_bytes = HD * elem_bytes(a.out_dt);
    for (int at = first * row_bytes + lane * 16; at < min(last, a.n_heads) * row_bytes; at += 512)
      *reinterpret_cast<uint4*>(ro + at) = make_uint4(0, 0, 0, 0);
    return;
  }
  const bool turned = u < a.turned;
  float2 cs[4], sn[4], ns[4];  // this lane's angles
  if (turned) {
    const int64_t at = pos * (a.turned * 8) + u * 8;
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(a.cos + at + 2 * e)), y = __ldg(reinterpret_cast<const float4*>(a.sin + at + 2 * e));
      cs[e] = make_float2(x.x, x.y), cs[e + 1] = make_float2(x.z, x.w);
      sn[e] = make_float2(y.x, y.y), sn[e + 1] = make_float2(y.z, y.w);
      ns[e] = make_float2(-y.x, -y.y), ns[e + 1] = make_float2(-y.z, -y.w);
    }
  }
  const int slot = (int)(pos & ((1 << c.log2_page) - 1));
  const int head_step = (HD * elem_bytes(CDT)) << c.log2_page;  // (32 bits hold it, as in the other rows' kernels)
  const int64_t cell0 = (int64_t)page * c.page_bytes + (int64_t)slot * (HD * elem_bytes(CDT));
  const int64_t scale0 = CDT == DT_E4M3 ? (int64_t)page * c.scale_stride + slot : 0;
  auto pairs = [](const float (&x)[8], float2 (&y)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = make_float2(x[2 * e], x[2 * e + 1]);
  };
  auto gains = [&](const uint8_t* g, int p, float2 (&y)[4]) {
    float x[8];
    if (a.gain_dt == DT_F32) {
      const float4 s = __ldg(reinterpret_cast<const float4*>(g) + 2 * p), t = __ldg(reinterpret_cast<const float4*>(g) + 2 * p + 1);
      x[0] = s.x, x[1] = s.y, x[2] = s.z, x[3] = s.w, x[4] = t.x, x[5] = t.y, x[6] = t.z, x[7] = t.w;
    } else if (a.gain_dt == DT_BF16) {
      load8<DT_BF16>(g + p * 16, x);
    } else {
      load8<DT_F16>(g + p * 16, x);
    }
    pairs(x, y);
  };
  const uint8_t* held = nullptr;  // whose gains this lane has
  float2 g[2][4];
#pragma unroll 1
  for (int h0 = first; h0 < last; h0 += kAhead * HPS) {
    if (h0 > first) load_rows(h0);
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      if (h0 + n * HPS >= last) break;
      const int h = h0 + n * HPS + lane / LPH, hk = h - a.n_heads, hv = hk - c.n_kv_heads;
      const bool on = h < last, is_q = hk < 0, is_v = hv >= 0;
      float2 x[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float y[8];
        raw[n][k].expand(y);
        pairs(y, x[k]);
      }
      if (!is_v) {
        const uint8_t* gain = is_q ? a.q_gain : a.k_gain;
        if (gain) {  // (all lanes of a head alike)
          if (gain != held) {
            gains(gain, pa, g[0]);
            gains(gain, pb, g[1]);
            held = gain;
          }
          const uint32_t mates = (LPH == 32 ? ~0u : (1u << LPH) - 1) << (lane / LPH * LPH);
          auto mean_square = [&]() {
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) sum = __ffma2_rn(x[k][e], x[k][e], sum);
            float ss = sum.x + sum.y;
#pragma unroll
            for (int d = LPH / 2; d >= 1; d >>= 1) ss += __shfl_xor_sync(mates, ss, d);
            return ss * (1.0f / HD);
          };
          float f = mean_square() + a.eps;
          if (!(f >= kLeastMean && f < INFINITY)) {
            // (rare) squares leave fp32's range: the head and eps are scaled by a power of two that brings the larger of them near 1
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) top = fmaxf(fmaxf(top, fabsf(x[k][e].x)), fabsf(x[k][e].y));
#pragma unroll
            for (int d = LPH / 2; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(mates, top, d));
            const float s = power_near(top, a.eps);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[k][e] = __fmul2_rn(x[k][e], make_float2(s, s));
            f = mean_square() + a.eps * s * s;
          }
          f = rsqrtf(f);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[k][e] = __fmul2_rn(__fmul2_rn(x[k][e], make_float2(f, f)), g[k][e]);
          }
        }
        if (turned) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 p = x[0][e], q = x[1][e];
            x[0][e] = __ffma2_rn(p, cs[e], __fmul2_rn(q, ns[e]));
            x[1][e] = __ffma2_rn(q, cs[e], __fmul2_rn(p, sn[e]));
          }
        }
      }
      if (!on) continue;
      if (is_q) {
        uint8_t* p = ro + h * HD * elem_bytes(a.out_dt);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int at = k ? pb : pa;
          float y[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[2 * e] = x[k][e].x, y[2 * e + 1] = x[k][e].y;
          if (a.out_dt == DT_BF16) store_row8<DT_BF16>(p + at * 16, y);
          else if (a.out_dt == DT_F16) store_row8<DT_F16>(p + at * 16, y);
          else store_row8<DT_F32>(p + at * 32, y);
        }
      } else {
        const int hc = is_v ? hv : hk;
        uint8_t* cell = (is_v ? c.v : c.k) + cell0 + hc * head_step;
        if constexpr (CDT == DT_E4M3) {
          float top = 0.0f;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max_nan(max_nan(top, fabsf(x[k][e].x)), fabsf(x[k][e].y));
          const uint32_t mates = (LPH == 32 ? ~0u : (1u << LPH) - 1) << (lane / LPH * LPH);
#pragma unroll
          for (int d = LPH / 2; d >= 1; d >>= 1) top = max_nan(top, __shfl_xor_sync(mates, top, d));
          const float s = quantise16(x, top);
          if (u == 0) (is_v ? c.v_scale : c.k_scale)[scale0 + ((int64_t)hc << c.log2_page)] = s;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[2 * e] = x[k][e].x, y[2 * e + 1] = x[k][e].y;
          store_row8<CDT>(cell + (k ? pb : pa) * 8 * elem_bytes(CDT), y);
        }
      }
    }
  }
}

// Launches one instance: a row's line of heads is cut over warps while all of the call's warps run at once (4 rows of 20 + 8
// heads: 2.6 us in a captured graph, 4.3 uncut; many rows gain nothing by it: 34,360 rows 137 us, 147 in halves, 198 in sixths).
// An SM holds 16 of these warps (four of up to 128 registers a thread on each of its quarters).  Cut by 24, calls of 2 rows
// of 32 + 16 bf16 heads an SM took 5.1 us instead of 3.5 and 12 rows an SM 8.8 instead of 7.1, some of their warps in a second
// round; by 12, 8 rows an SM 6.3 instead of 5.6.
template <int ROWDT, int CDT, int HD>
cudaError_t append_launch(AppendArgs& a, int sms, cudaStream_t st) {
  auto* kernel = paged_append_kernel<ROWDT, CDT, HD>;
  static int known[64];  // warps that an SM of a device holds
  int dev = 0, held = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64) held = known[dev];
  if (!held) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&held, kernel, kAppendThreads, 0);
    if (e != cudaSuccess) return e;
    held *= kAppendThreads / 32;
    if (dev < 64) known[dev] = held;
  }
  const int heads = a.n_heads + 2 * a.c.n_kv_heads;
  a.part_heads = row_part_heads(heads, 32 / (HD / 16), a.n_rows, sms * held);
  a.parts = (heads + a.part_heads - 1) / a.part_heads;
  const int64_t grid = ((int64_t)a.n_rows * a.parts + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  kernel<<<(unsigned)grid, kAppendThreads, 0, st>>>(a);
  return cudaGetLastError();
}

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
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaSuccess;
  auto by_rows = [&](auto cdt, auto hd) {
    constexpr int C = decltype(cdt)::value, H = decltype(hd)::value;
    if (rows_dtype == ADP_F16) e = append_launch<DT_F16, C, H>(a, sms, st);
    else if (rows_dtype == ADP_BF16) e = append_launch<DT_BF16, C, H>(a, sms, st);
    else e = append_launch<DT_F32, C, H>(a, sms, st);
  };
  auto by_cache = [&](auto hd) {
    if (kv->dtype == ADP_F16) by_rows(std::integral_constant<int, DT_F16>(), hd);
    else if (kv->dtype == ADP_BF16) by_rows(std::integral_constant<int, DT_BF16>(), hd);
    else by_rows(std::integral_constant<int, DT_E4M3>(), hd);
  };
  if (kv->head_dim == 128) by_cache(std::integral_constant<int, 128>());
  else by_cache(std::integral_constant<int, 64>());
  return cuda_status(e, "adp_paged_kv_append");
}
