// Causal attention of packed prompts on the tensor cores.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "../../include/adp.h"
#include "device.cuh"
#include "paged.cuh"
#include "tc.cuh"

namespace adp {
namespace {

constexpr int kRows = 128;            // rows of a query tile (M of the MMA), and keys of a block
constexpr int kThreads = 384;         // 8 softmax warps, the copying and the issuing warp, two idle ones
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr float kRescale = 8.0f;      // base-2 growth of a row's maximum that rescales its output

struct PackedArgs {
  const int32_t* cu_q;
  const int32_t* cu_k;
  const uint8_t* v;
  uint8_t* out;
  int64_t v_stride, out_stride;  // bytes
  int32_t n_seqs, n_q, n_k, hkv, group, tok;
  float scale_log2;              // of |scale|
  int32_t negative;              // scale < 0
  int32_t* status;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A sequence's rows [begin, begin + n) of a packed tensor of `total` rows.
__device__ __forceinline__ void packed_range(const int32_t* cu, int b, int total, int32_t* status, int* begin, int* n) {
  const int a = cu[b], e = cu[b + 1];
  const int lo = min(max(a, 0), total), hi = min(max(e, lo), total);
  if (lo != a || hi != e) report(status, ADP_ERR_INVALID_ARG);
  *begin = lo;
  *n = hi - lo;
}

template <int HD>
struct PackedSmem {
  static constexpr int kSlots = HD == 128 ? 5 : 8;
  static constexpr uint32_t kBlock = 128 * 128;             // 128 rows x 64 elements, swizzled
  static constexpr uint32_t kTile = (HD / 64) * kBlock;     // 128 rows of Q, K or V
  static constexpr uint32_t kBars = (2 + kSlots) * kTile;   // Q tiles, ring, then the barriers
  static constexpr size_t kBytes = 1024 + kBars + 512;
};

// CTA: one KV head's group of query heads for 2 x tok consecutive tokens of one sequence, as two tiles A and B of 128
// rows (row = token x group + head: tok = 128 / group tokens, so a group's heads share K and V and the causal edge is
// only tok tokens wide).  Three warpgroups: warps 0-3 the softmax of tile A, 4-7 of tile B (thread = row = TMEM lane),
// warp 8 copies, warp 9 issues the MMAs.
//  - copies: both Q tiles, then K and V blocks of 128 keys in turn into a ring of 32 KB slots (128-byte swizzled);
//  - S = Q K^T per tile into 128 TMEM columns; the softmax reads S, writes P (16-bit) over it, and O += P V takes P from
//    TMEM and V as the MN-major operand.  The two tiles alternate: while A's softmax runs the tensor cores work on B.
//    One thread issues all MMAs in the order PV_A(j) S_A(j+1) PV_B(j) S_B(j+1), so S_A(j+1)'s completion also says that
//    PV_A(j) is done: O may be rescaled then, and P has been read;
//  - a row's running maximum is replaced only when it grows by more than 2^8 (decided per warp): O and the sum carry the
//    same stale factor, which cancels.
// TMEM: S/P of A and B (128 columns each), O of A and B (HD columns each).
// Keys that a row does not see: their scores are replaced; their V must not meet the zero probabilities if it is not
// finite, so blocks on the causal edge or the sequence's end are looked through in shared memory: rows behind the
// sequence become zeros, non-finite elements too, and the (rare) latter are added to the rows that do see them at the end.
template <int HD, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    packed_attention_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                            const __grid_constant__ CUtensorMap mv, const PackedArgs a) {
  using L = PackedSmem<HD>;
  constexpr int NS = L::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* Qs = smem;
  uint8_t* ring = smem + 2 * L::kTile;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* qfull = bar;
  uint64_t* full = bar + 1;           // [NS]
  uint64_t* empty = full + NS;        // [NS]
  uint64_t* sfull = empty + NS;       // [2]
  uint64_t* pready = sfull + 2;       // [2]
  uint64_t* odone = pready + 2;       // [2]
  uint64_t* done = odone + 2;
  int32_t* ctl = reinterpret_cast<int32_t*>(done + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctl);
  volatile int32_t* ab = ctl + 1;
  volatile int32_t* bad = ctl + 2;    // a non-finite value was taken out of an edge block
  int32_t* item = ctl + 3;            // [6]: sequence's first query row, queries, first key row, keys, first token, found
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x % a.hkv;
  const int span = 2 * a.tok;

  if (threadIdx.x == 0) {
    mbar_init(qfull, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sfull[t], 1);
      mbar_init(&pready[t], 128);
      mbar_init(&odone[t], 1);
    }
    mbar_init(done, 1);
    *ab = 0;
    *bad = 0;
    mbar_fence_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 8) {
    // this CTA's tokens: pair r of all sequences' pairs, the last of each sequence first (they see the most keys)
    int r = blockIdx.x / a.hkv;
    if (lane == 0) item[5] = 0;
    __syncwarp();
    for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
      int q0 = 0, nq = 0;
      if (b0 + lane < a.n_seqs) packed_range(a.cu_q, b0 + lane, a.n_q, a.status, &q0, &nq);
      const int pairs = (nq + span - 1) / span;
      int sum = pairs;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += o;
      }
      const int all = __shfl_sync(0xFFFFFFFFu, sum, 31);
      if (r < all) {
        if (r < sum && r >= sum - pairs) {
          int k0, nk;
          packed_range(a.cu_k, b0 + lane, a.n_k, a.status, &k0, &nk);
          item[0] = q0, item[1] = nq, item[2] = k0, item[3] = nk;
          item[4] = (pairs - 1 - (r - (sum - pairs))) * span;
          item[5] = 1;
        }
        break;
      }
      r -= all;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool work = item[5] != 0;
  const int q0 = item[0], lq = item[1], k0 = item[2], lk = item[3], t0 = item[4];
  const int off = lk - lq;
  // key blocks that each tile's last token sees
  int nk[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = t0 + t * a.tok, last = min(first + a.tok, lq) - 1;
    nk[t] = work && first < lq && last + off >= 0 ? (last + off) / kRows + 1 : 0;
  }
  const int n = max(nk[0], nk[1]);
  int32_t never = 0;

  // A softmax thread holds a row of 128 scores: its warpgroups take registers that the third one gives back
  // (256 x 208 + 128 x 80 = 63,488 of the 384 x 168 = 64,512 that the block is launched with).
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 8) {
      if (lane == 0 && n > 0) {
        const uint32_t qbytes = (uint32_t)(a.tok * a.group) * 128 * (HD / 64);
        int issued = 0;
        const int tiles = nk[1] > 0 ? 2 : 1;
        mbar_arrive_expect_tx(qfull, qbytes * tiles);
        for (int t = 0; t < tiles; ++t)
          for (int c = 0; c < HD / 64; ++c)
            tma_load_3d(Qs + t * L::kTile + c * L::kBlock, &mq, c * 64, h * a.group, q0 + t0 + t * a.tok, qfull);
        for (int i = 0; i < 2 * n; ++i) {
          const int s = i % NS;
          if (i >= NS && !mbar_wait(&empty[s], (i / NS - 1) & 1, ab, kWaitNs)) {
            *ab = 1;
            break;
          }
          mbar_arrive_expect_tx(&full[s], L::kTile);
          for (int c = 0; c < HD / 64; ++c)
            tma_load_3d(ring + s * L::kTile + c * L::kBlock, i & 1 ? &mv : &mk, c * 64, h, k0 + (i >> 1) * kRows, &full[s]);
          issued = i + 1;
        }
        // no copy may still be writing this CTA's shared memory when it exits
        mbar_wait(qfull, 0, &never, kWaitNs);
        for (int i = issued > NS ? issued - NS : 0; i < issued; ++i) mbar_wait(&full[i % NS], (i / NS) & 1, &never, kWaitNs);
      }
      __syncwarp();
    } else if (warp == 9) {
      if (lane == 0) {
        constexpr uint32_t id_s = tc_idesc_f16(BF16, 128, 128);
        constexpr uint32_t id_o = tc_idesc_f16(BF16, 128, HD) | kTcIdescBMn;
        const uint32_t q_addr = smem_u32(Qs), ring_addr = smem_u32(ring);
        auto score = [&](int t, int j) -> bool {
          const int i = 2 * j, s = i % NS;
          if (!mbar_wait(&full[s], (i / NS) & 1, ab, kWaitNs)) return false;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint32_t at = (k / 4) * L::kBlock + (k % 4) * 32;
            tc_mma_f16(tmem + t * 128, tc_smem_desc_sw128(q_addr + t * L::kTile + at, 16, 1024),
                       tc_smem_desc_sw128(ring_addr + s * L::kTile + at, 16, 1024), id_s, k > 0);
          }
          tc_commit(&sfull[t]);
          return true;
        };
        auto weigh = [&](int t, int j) -> bool {
          const int i = 2 * j + 1, s = i % NS;
          if (!mbar_wait(&full[s], (i / NS) & 1, ab, kWaitNs) || !mbar_wait(&pready[t], j & 1, ab, kWaitNs)) return false;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_f16_ts(tmem + 256 + t * 128, tmem + t * 128 + k * 8,
                          tc_smem_desc_sw128(ring_addr + s * L::kTile + k * 2048, L::kBlock, 1024), id_o, j > 0 || k > 0);
          return true;
        };
        bool ok = true;
        if (n > 0) {
          ok = mbar_wait(qfull, 0, ab, kWaitNs);
          for (int t = 0; t < 2; ++t)
            if (ok && nk[t] > 0) ok = score(t, 0);
          if (ok) tc_commit(&empty[0]);
        }
        for (int j = 0; ok && j < n; ++j) {
          for (int t = 0; ok && t < 2; ++t) {
            if (j >= nk[t]) continue;
            ok = weigh(t, j);
            if (!ok) break;
            if (t == 1 || j >= nk[1]) tc_commit(&empty[(2 * j + 1) % NS]);  // the block's last use
            if (j + 1 == nk[t]) tc_commit(&odone[t]);
            if (j + 1 < nk[t]) {
              ok = score(t, j + 1);
              if (ok && (t == 1 || j + 1 >= nk[1])) tc_commit(&empty[(2 * j + 2) % NS]);
            }
          }
        }
        if (!ok) *ab = 1;
        tc_commit(done);  // on every path: arrives once no MMA of this CTA is in flight
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = warp >> 2, r = threadIdx.x & 127;
    const int tok = t0 + t * a.tok + r / a.group, head = h * a.group + r % a.group;
    const bool live = work && r < a.tok * a.group && tok < lq;
    const int lim = min(tok + off, lk - 1);  // the last key that this row sees
    // the first key that some row of the CTA's tiles does not see: from its block on, blocks are edge blocks
    const int edge_a = t0 + off + 1, edge_b = t0 + a.tok + off + 1;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + t * 128, tO = tmem + lanes + 256 + t * 128;
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    auto wait_all = [&](uint64_t* b, uint32_t parity) {
      return __all_sync(0xFFFFFFFFu, mbar_wait(b, parity, ab, kWaitNs));
    };
    for (int j = 0; j < nk[t]; ++j) {
      if (!wait_all(&sfull[t], j & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float x[128];
      tmem_ld128(tS, x);
      if (a.negative) {
#pragma unroll
        for (int c = 0; c < 128; ++c) x[c] = -x[c];
      }
      const int left = lim - j * kRows;  // columns c <= left are seen
      const bool all_seen = __all_sync(0xFFFFFFFFu, left >= 127);
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (!all_seen) {
#pragma unroll
        for (int c = 0; c < 128; ++c) x[c] = c <= left ? x[c] : -INFINITY;
      }
#pragma unroll
      for (int c = 0; c < 128; ++c) top[c & 3] = fmaxf(top[c & 3], x[c]);
      const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      const float mb = mx == -INFINITY ? -INFINITY : mx * a.scale_log2;
      const bool grow = mb > m + kRescale || (m == -INFINITY && mb > -INFINITY);
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float mn = fmaxf(m, mb);
        const float f = mn == -INFINITY ? 1.0f : exp2_fast(m - mn);
        m = mn;
        l *= f;
        if (j > 0) {
#pragma unroll
          for (int c0 = 0; c0 < HD; c0 += 32) {
            float o[32];
            tmem_ld32(tO + c0, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f;
            tmem_st32(tO + c0, o);
          }
        }
      }
      const float ms = m == -INFINITY ? 0.0f : m;
      const float2 sc = make_float2(a.scale_log2, a.scale_log2), nm = make_float2(-ms, -ms);
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
      for (int c0 = 0; c0 < 128; c0 += 32) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 y = __ffma2_rn(make_float2(x[c0 + e], x[c0 + e + 1]), sc, nm);
          float2 p = make_float2(exp2_fast(y.x), exp2_fast(y.y));
          if (!all_seen) {
            p.x = c0 + e <= left ? p.x : 0.0f;
            p.y = c0 + e + 1 <= left ? p.y : 0.0f;
          }
          sum[(e >> 1) & 1] = __fadd2_rn(sum[(e >> 1) & 1], p);
          w[e >> 1] = pack2(p.x, p.y, BF16 ? DT_BF16 : DT_F16);
        }
        tmem_st16(tS + c0 / 2, w);
      }
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      // ---- an edge block's values, looked through by the first tile that takes it
      if ((t == 0 || j >= nk[0]) && (j + 1) * kRows > (j < nk[0] ? edge_a : edge_b)) {
        const int i = 2 * j + 1, s = i % NS;
        if (!wait_all(&full[s], (i / NS) & 1)) {
          ok = false;
          break;
        }
        const bool outside = j * kRows + r >= lk;
#pragma unroll 1
        for (int c = 0; c < HD / 8; ++c) {
          uint4* p = reinterpret_cast<uint4*>(ring + s * L::kTile + (c / 8) * L::kBlock + r * 128 + (((c & 7) ^ (r & 7)) * 16));
          uint4 v = outside ? make_uint4(0, 0, 0, 0) : *p;
          constexpr uint32_t kExp = BF16 ? 0x7F80u : 0x7C00u;
          bool odd = false;
          uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool lo = (w[e] & kExp) == kExp, hi = (w[e] & (kExp << 16)) == (kExp << 16);
            odd |= lo | hi;
            w[e] = (lo ? 0u : w[e] & 0xFFFFu) | (hi ? 0u : w[e] & 0xFFFF0000u);
          }
          if (odd) *bad = 1;
          if (odd || outside) *p = v;
        }
        fence_async_smem();
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&pready[t]);
    }
    // ---- O / l
    if (nk[t] > 0 && ok) ok = wait_all(&odone[t], 0);
    tc_fence_after();
    if (ok) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      uint8_t* po = a.out + (int64_t)(q0 + tok) * a.out_stride + (int64_t)head * HD * 2;
#pragma unroll
      for (int c0 = 0; c0 < HD; c0 += 32) {
        float o[32];
        if (nk[t] > 0) {
          tmem_ld32(tO + c0, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.0f;
        }
        if (!live) continue;
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = l == 0.0f ? 0.0f : o[e] * inv;
        if (*bad) {
          for (int key = max(0, edge_a / kRows * kRows); key <= lim; ++key) {
            const uint8_t* pv = a.v + (int64_t)(k0 + key) * a.v_stride + (int64_t)h * HD * 2 + c0 * 2;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint32_t bits = reinterpret_cast<const uint16_t*>(pv)[e];
              const float v = kv_to_f32((uint16_t)bits, BF16 ? DT_BF16 : DT_F16);
              o[e] += isfinite(v) ? 0.0f : v;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = pack2(o[e + 2 * k], o[e + 2 * k + 1], BF16 ? DT_BF16 : DT_F16);
          *reinterpret_cast<uint4*>(po + (c0 + e) * 2) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    } else {
      *ab = 1;
      if (r == 0) report(a.status, ADP_ERR_PIPELINE_TIMEOUT);
    }
  }
  // no MMA may be in flight (nor TMEM in use) when the accumulators are freed
  mbar_wait(done, 0, &never, kWaitNs);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- host side

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// [rows][heads][hd] of 16-bit elements, boxes of 64 elements x box_heads x box_rows.
bool encode(CUtensorMap* map, const void* base, bool bf16, int hd, int heads, int64_t rows, int64_t stride, int box_heads,
            int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)hd, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)hd * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, one[3] = {1, 1, 1};
  return encode_fn()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                     const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, bool BF16>
struct PackedKey {};

template <int HD, bool BF16>
cudaError_t packed_launch(const CUtensorMap (&m)[3], const PackedArgs& a, int64_t grid, cudaStream_t st) {
  auto* kernel = packed_attention_kernel<HD, BF16>;
  const cudaError_t e = allow_smem<PackedKey<HD, BF16>>((const void*)kernel, PackedSmem<HD>::kBytes);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)grid, kThreads, PackedSmem<HD>::kBytes, st>>>(m[0], m[1], m[2], a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace adp

using namespace adp;

extern "C" int adp_packed_attention(const void* q, const void* k, const void* v, int32_t dtype, int32_t n_heads,
                                    int32_t n_kv_heads, int32_t head_dim, int64_t q_stride, int64_t k_stride,
                                    int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k, int32_t n_seqs,
                                    int32_t n_q, int32_t n_k, float scale, void* out, int64_t out_stride,
                                    int32_t* dev_status, void* cuda_stream) {
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || n_seqs < 0 || n_q < 0 || n_k < 0 || !isfinite(scale))
    return ADP_ERR_INVALID_ARG;
  if (dtype != ADP_F16 && dtype != ADP_BF16) return ADP_ERR_UNSUPPORTED_CONFIG;
  if (head_dim != 64 && head_dim != 128) return ADP_ERR_UNSUPPORTED_CONFIG;
  const int group = n_heads / n_kv_heads;
  if (group > kRows || n_heads > 65536) return ADP_ERR_UNSUPPORTED_CONFIG;
  if (((uintptr_t)cu_q | (uintptr_t)cu_k | (uintptr_t)dev_status) & 3) return ADP_ERR_INVALID_ARG;
  if (n_seqs == 0 || n_q == 0) return ADP_OK;
  if (!cu_q || !cu_k || !q || !out || !aligned16(q) || !aligned16(out)) return ADP_ERR_INVALID_ARG;
  const int64_t qw = (int64_t)n_heads * head_dim, kw = (int64_t)n_kv_heads * head_dim;
  if (q_stride < qw || out_stride < qw || q_stride % 8 || out_stride % 8) return ADP_ERR_INVALID_ARG;
  if (n_k > 0 && (!k || !v || !aligned16(k) || !aligned16(v) || k_stride < kw || v_stride < kw || k_stride % 8 || v_stride % 8))
    return ADP_ERR_INVALID_ARG;
  if (!encode_fn()) return cuda_status(cudaErrorNotSupported, "cuTensorMapEncodeTiled");
  const bool bf16 = dtype == ADP_BF16;
  const int tok = kRows / group;
  CUtensorMap m[3];
  // (without keys no block is copied, and the maps of K and V are any valid ones)
  if (!encode(&m[0], q, bf16, head_dim, n_heads, n_q, q_stride, group, tok) ||
      !encode(&m[1], n_k ? k : q, bf16, head_dim, n_kv_heads, n_k ? n_k : 1, n_k ? k_stride : kw, 1, kRows) ||
      !encode(&m[2], n_k ? v : q, bf16, head_dim, n_kv_heads, n_k ? n_k : 1, n_k ? v_stride : kw, 1, kRows))
    return ADP_ERR_INVALID_ARG;
  PackedArgs a{cu_q, cu_k, static_cast<const uint8_t*>(v), static_cast<uint8_t*>(out), v_stride * 2, out_stride * 2,
               n_seqs, n_q, n_k, n_kv_heads, group, tok, fabsf(scale) * 1.4426950408889634f, scale < 0.0f, dev_status};
  const int64_t pairs = (int64_t)n_q / (2 * tok) + n_seqs;  // at most: every sequence may end inside a pair
  const int64_t grid = pairs * n_kv_heads;
  if (grid > 0x7FFFFFFF) return ADP_ERR_UNSUPPORTED_CONFIG;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e;
  if (head_dim == 128) e = bf16 ? packed_launch<128, true>(m, a, grid, st) : packed_launch<128, false>(m, a, grid, st);
  else e = bf16 ? packed_launch<64, true>(m, a, grid, st) : packed_launch<64, false>(m, a, grid, st);
  return cuda_status(e, "adp_packed_attention");
}
