// Attention of one new token per sequence over the pages of a KV cache, over all of its positions or those that a window and
// the first positions leave.
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>

#include <type_traits>

#include "../../include/adp.h"
#include "device.cuh"
#include "paged.cuh"

namespace adp {
namespace {

__device__ __forceinline__ uint4 ldg16(const uint8_t* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg8(const uint8_t* p) {
  uint2 v;
  asm("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// D += A B on the warp-level tensor instruction, 16 x 16 by 16 x 8, fp32 accumulators.
template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (BF16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}
// Transpose of an 8 x 8 matrix of 16-bit elements held by a warp (row lane / 4, columns 2 (lane % 4) and + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Four e4m3 codes as fp16 (exact): the low pair and the high pair.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
constexpr float kStale = 8.0f;  // how far scores may exceed the maximum in use (base-2 exponents)
constexpr float kFactorMax = 1.329227996e36f;  // 2^120, of a value scale relative to the largest product
// fp16 weights are held 2^7 times larger, and their sum alike: up to 2^15 beside a stale maximum they fit, and a weight has
// all its bits down to 2^-21 of the largest and some down to 2^-32, so that a long context's tail does not vanish beside
// one dominating position.  (bf16 has fp32's range.)
template <int CDT>
constexpr float kWeightUp = CDT == DT_BF16 ? 0.0f : 7.0f;

__device__ __forceinline__ float safe_max(float m) { return m == -INFINITY ? 0.0f : m; }

// Softmax state of a piece of a segment, in shared or global memory.
template <int HD, int NT>
struct Partial {
  float o[NT * 8][HD];
  float m[NT * 8];
  float l[NT * 8];
};
struct SplitMeta {
  int32_t seg;   // sequence x tile of heads that starts in this CTA and goes on behind it, -1: none
  int32_t last;  // the CTA that it ends in
};

struct AttnArgs {
  PagedView c;
  const uint8_t* q;
  uint8_t* out;
  int64_t q_stride, out_stride;  // bytes
  int32_t group, tiles;          // query heads per KV head; tiles of query heads per KV head
  float scale_log2;
  void* partials;                // Partial [2 ctas]
  SplitMeta* meta;               // [ctas]
  int32_t* status;
  int32_t cluster;               // CTAs per segment (a cluster), 0: the line of all units is cut evenly
  int32_t window, sinks;         // (only with a window) the last positions that are seen, and the first
};

// What a sequence's new token sees in units of UNIT positions: those of the first `sinks` positions and those of the last
// `window`, one line without the units between them.  (The line is what is cut, so that a
// call costs what its window leaves: 64 sequences of up to 16,000 positions in e4m3, window 4,096: 96 us, 74% of the copy rate; one of
// 131,000 in bf16, window 32,768: 35 us, 57%, start and join about 12 us of it.)
template <int UNIT>
struct Seen {
  int len, first, low, head, gap;  // positions: length, sinks in front of the window, the window's first; units of the sinks, and left out
  __device__ __forceinline__ Seen(int l, int window, int sinks) : len(l) {
    low = len > window ? len - window : 0;
    first = sinks < low ? sinks : low;
    head = (first + UNIT - 1) / UNIT;
    gap = low / UNIT > head ? low / UNIT - head : 0;
  }
  __device__ __forceinline__ int units() const { return (len + UNIT - 1) / UNIT - gap; }
  __device__ __forceinline__ int unit(int t) const { return t < head ? t : t + gap; }
  __device__ __forceinline__ bool sees(int pos) const { return pos < len && (pos >= low || pos < first); }
  // whether some of, and whether all n positions from pos on are seen
  __device__ __forceinline__ bool any(int pos, int n) const { return pos < len && (pos + n > low || pos < first); }
  __device__ __forceinline__ bool all(int pos, int n) const { return pos + n <= len && (pos >= low || pos + n <= first); }
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Loads from the shared memory of CTA `rank` of the cluster, at this CTA's address p.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_u32(p)), "r"(rank));
  return d;
}
__device__ __forceinline__ float cluster_ld(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// CTAs per SM: 12 warps of 168 registers, or 8 of 255 for the wider tile of heads.
template <int NT>
constexpr int kResident = NT == 1 ? 3 : 2;

// One new token per sequence over its pages.  The line of units (a unit: 4 KB of keys, i.e. 16 to 64 positions, of
// one sequence, KV head and tile of up to 8 NT query heads) is cut into even ranges, one per CTA and in it one per
// warp, whatever the sequences' lengths are: a long context spreads over the GPU and short ones share a warp.
// A warp runs its range segment by segment (segment: one sequence and tile of heads) with its own running maximum,
// sum and output in registers.  Segments that several warps share are joined in shared memory, segments that
// several CTAs share in paged_attention_join_kernel.
// Where every segment is short and there are few (a.cluster), each gets a cluster of 1 to 8 CTAs instead, whose warps
// share its units and join through distributed shared memory: no sums over the lengths, no workspace and no second
// launch, which is what small calls wait for.
//
// Bound by reading K and V once.  Both go from global memory straight into the registers of the 16 x 8 x 16 tensor
// instruction: S^T = K Q^T takes a K row's 16-byte pieces as the A operand (the order of the contraction index is
// free, and Q's is chosen alike), O^T = V^T P^T takes V's with the 16-bit halves of two keys interleaved.  With the
// query heads as the 8-wide side a group of up to 8 heads costs one instruction per 16 x 16 of K; nothing is staged
// in shared memory.  e4m3 codes become fp16 (exact), their scales multiply the scores and the probabilities.
// Measured: 131,011 bf16 positions of 8 KV heads 91.5 us (5.9 TB/s), 64 ragged e4m3 sequences 87 us (5.2 TB/s; the same
// with one unit of O for a warp, the largest value scale, which took bits from the others whatever its own weight; head_dim 64
// 65 us instead of 61); with an
// L2 prefetch of one unit more 96 and 93.  The first form (8 warps, every load predicated, a maximum updated every unit)
// took 124 us for the latter.
template <int HD, int CDT, int QDT, int NT, bool SMALL, bool WIN>
__global__ void __launch_bounds__(kPagedWarps * 32, kResident<NT>) paged_attention_kernel(AttnArgs a) {
  constexpr int EB = elem_bytes(CDT);
  constexpr int ROWB = HD * EB;
  constexpr int UNIT = 4096 / ROWB;  // positions
  constexpr int RG = UNIT / 16;      // groups of 16 positions
  constexpr int KC = ROWB / 64;      // 16-byte pieces of a K row per lane
  constexpr int KS = 4 / EB;         // contraction steps per piece (a step: 4 elements per lane)
  constexpr int VB = ROWB / 8;       // bytes of a V row per lane
  constexpr int VW = VB / 4;         // 32-bit words
  constexpr int MT = HD / 16;        // 16-row tiles of O^T
  constexpr bool Q8 = CDT == DT_E4M3;
  constexpr bool BF = CDT == DT_BF16;  // type of the tensor instruction (e4m3: fp16)
  using Part = Partial<HD, NT>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Part* slots = reinterpret_cast<Part*>(smem_raw);  // [warps][2]
  __shared__ int32_t s_seg[kPagedWarps * 2];
  __shared__ int64_t s_u0[kPagedWarps * 2], s_u1[kPagedWarps * 2];
  __shared__ int64_t s_chunk[kPagedMaxSeqs / 32 + 1];
  const PagedView& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l4 = lane & 3, r8 = lane >> 2;
  const int nvt = c.n_kv_heads * a.tiles;

  auto units_in = [&](int len) {
    if constexpr (WIN) return Seen<UNIT>(len, a.window, a.sinks).units();
    else return (len + UNIT - 1) / UNIT;
  };
  auto units_of = [&](int b) { return units_in(paged_length(c.lens[b], c.table_width, c.log2_page)); };
  const int n_chunks = (c.n_seqs + 31) / 32;
  int64_t u, u_end, c0 = 0, c1 = 0, total = 0;
  int parts = 1, b = 0, vt = 0, t = 0, seg_units = 0;
  if (threadIdx.x < kPagedWarps * 2) s_seg[threadIdx.x] = -1;
  __syncthreads();
  if (a.cluster) {
    const int seg = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
    b = seg / nvt;
    vt = seg % nvt;
    const int32_t raw = c.lens[b], len = paged_length(raw, c.table_width, c.log2_page);
    if (raw > len) report(a.status, ADP_ERR_CONTEXT_OVERFLOW);
    if (raw < 0) report(a.status, ADP_ERR_INVALID_ARG);
    seg_units = units_in(len);
    const int w = rank * kPagedWarps + warp;
    t = (int)((uint32_t)seg_units * w / (uint32_t)(a.cluster * kPagedWarps));  // (few units: no overflow)
    u = t;
    u_end = (uint32_t)seg_units * (w + 1) / (uint32_t)(a.cluster * kPagedWarps);
  } else {
    // ---- the line's length: units of every 32 sequences, and zeros for the sequences without any
    for (int ch = warp; ch < n_chunks; ch += kPagedWarps) {
      const int b = ch * 32 + lane;
      int n = 0;
      bool empty = false;
      if (b < c.n_seqs) {
        const int32_t raw = c.lens[b], len = paged_length(raw, c.table_width, c.log2_page);
        if (raw > len) report(a.status, ADP_ERR_CONTEXT_OVERFLOW);
        if (raw < 0) report(a.status, ADP_ERR_INVALID_ARG);
        n = units_in(len);
        empty = n == 0 && b % gridDim.x == blockIdx.x;
      }
      for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, empty); todo; todo &= todo - 1) {
        uint8_t* o = a.out + (int64_t)(ch * 32 + __ffs(todo) - 1) * a.out_stride;
        const int words = c.n_kv_heads * a.group * HD / 8;
        for (int w = lane; w < words; w += 32) reinterpret_cast<uint4*>(o)[w] = make_uint4(0, 0, 0, 0);
      }
      n = __reduce_add_sync(0xFFFFFFFFu, n);
      if (lane == 0) s_chunk[ch] = n;
    }
    __syncthreads();
    if (warp == 0) {  // running sums over the chunks, in place: s_chunk[i] = units before chunk i
      int64_t run = 0;
      for (int ch = 0; ch <= n_chunks; ch += 32) {
        int64_t n = ch + lane < n_chunks ? s_chunk[ch + lane] : 0, sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int64_t o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
          if (lane >= d) sum += o;
        }
        if (ch + lane <= n_chunks) s_chunk[ch + lane] = run + sum - n;
        run += __shfl_sync(0xFFFFFFFFu, sum, 31);
      }
    }
    __syncthreads();
    total = s_chunk[n_chunks] * nvt;
    parts = split_parts(total, gridDim.x);
    if ((int)blockIdx.x >= parts || total == 0) {
      if (threadIdx.x == 0) a.meta[blockIdx.x].seg = -1;
      return;
    }
    c0 = split_begin(total, parts, blockIdx.x);
    c1 = split_begin(total, parts, blockIdx.x + 1);
    u = c0 + split_begin(c1 - c0, kPagedWarps, warp);
    u_end = c0 + split_begin(c1 - c0, kPagedWarps, warp + 1);
  }
  const int64_t u_first = u;
  const int b0 = b, vt0 = vt;  // a cluster's segment

  if (u < u_end) {
    if (!a.cluster) {  // ---- the sequence, head tile and unit of u
      const int64_t seq_u = u / nvt;
      int ch = 0;
      for (int at = 0; at < n_chunks; at += 32) {
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, at + lane < n_chunks && s_chunk[at + lane] <= seq_u));
        if (n) ch = at + n - 1;
        if (n < 32) break;
      }
      const int bl = ch * 32 + lane;
      const int n = bl < c.n_seqs ? units_of(bl) : 0;
      int sum = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += o;
      }
      const int64_t rest = u - s_chunk[ch] * nvt;
      const int skip = __popc(__ballot_sync(0xFFFFFFFFu, (int64_t)sum * nvt <= rest));
      b = min(ch * 32 + skip, c.n_seqs - 1);
      const int nb = max(1, __shfl_sync(0xFFFFFFFFu, n, skip & 31));
      const int before = __shfl_sync(0xFFFFFFFFu, sum - n, skip & 31);
      const int64_t in = rest - (int64_t)before * nvt;
      vt = (int)(in / nb);
      t = (int)(in - (int64_t)vt * nb);
    }
    while (u < u_end) {
      const int len = paged_length(c.lens[b], c.table_width, c.log2_page);
      const Seen<UNIT> seen(len, WIN ? a.window : 0, WIN ? a.sinks : 0);  // (unused without a window)
      const int n_units = units_in(len);
      const int n = (int)min((int64_t)(n_units - t), u_end - u);
      if (n <= 0 || vt >= nvt) break;  // the lengths changed while this call ran
      const int kvh = vt / a.tiles, head0 = (vt % a.tiles) * (NT * 8);
      const int heads = min(NT * 8, a.group - head0);
      const int32_t* trow = c.table + (int64_t)b * c.table_width;

      // ---- the queries, as the B operand (columns: heads)
      uint32_t qf[NT][MT][2];
      float qs[NT][2];  // score factor of this lane's two columns
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int h = nt * 8 + r8;
        const uint8_t* qr = a.q + (int64_t)b * a.q_stride + (int64_t)(kvh * a.group + head0 + h) * HD * 2;
#pragma unroll
        for (int ks = 0; ks < MT; ++ks) {
          const int d = (ks / KS) * (64 / EB) + l4 * (16 / EB) + (ks % KS) * 4;
          const uint2 w = h < heads ? ldg8(qr + d * 2) : make_uint2(0, 0);
          qf[nt][ks][0] = w.x;
          qf[nt][ks][1] = w.y;
        }
        float f = 1.0f;
        if constexpr (Q8 && QDT == DT_BF16) {
          // bf16 queries meet fp16 codes: the row is brought to a largest magnitude in [1, 2) by a power of two,
          // so that its 8-bit significands fit fp16 (an element below 2^-17 loses bits: at most 2^-25, half fp16's
          // least step)
          float top = 0.0f;
#pragma unroll
          for (int ks = 0; ks < MT; ++ks)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qf[nt][ks][j] << 16)),
                                     fabsf(__uint_as_float(qf[nt][ks][j] & 0xFFFF0000u))));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const uint32_t e = min(max(__float_as_uint(top) >> 23, 1u), 253u);
          f = __uint_as_float(e << 23);
          const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
          for (int ks = 0; ks < MT; ++ks)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              qf[nt][ks][j] = pack2(__uint_as_float(qf[nt][ks][j] << 16) * inv,
                                    __uint_as_float(qf[nt][ks][j] & 0xFFFF0000u) * inv, DT_F16);
        }
        // this lane's scores are of heads 2 l4 and 2 l4 + 1, whose factors lanes 8 l4 and 8 l4 + 4 hold
        qs[nt][0] = __shfl_sync(0xFFFFFFFFu, f, l4 * 8) * a.scale_log2;
        qs[nt][1] = __shfl_sync(0xFFFFFFFFu, f, l4 * 8 + 4) * a.scale_log2;
      }

      float o[MT][NT][4];
      float m[NT][2], l[NT][2];
      // e4m3: what weighs V's codes are the products weight x value scale.  They have a running maximum of their own, mo
      // (base-2 exponents: score + log2 of the scale), O is relative to it, and vc = 2^(m - mo) brings them there: a large
      // scale counts only with its weight, so that one beside a negligible weight takes no bits from the others.
      float mo[NT][2], vc[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = mo[nt][0] = mo[nt][1] = -INFINITY;
        vc[nt][0] = vc[nt][1] = 1.0f;
        l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.0f;
      }

      uint32_t kr[RG][2][KC * 4];
      uint32_t vr[RG][4][VW];
      float ksc[RG][2], vsc[RG][2];
      const int in_page = (1 << c.log2_page) - 1;
      // Page of the n positions from pos on (all in one page) where one of them is attended, else -1.
      auto page_at = [&](int pos, int n) {
        if (WIN ? !seen.any(pos, n) : pos >= len) return -1;
        const int page = paged_page(trow, c.table_width, c.n_pages, c.log2_page, pos);
        if (page < 0) report(a.status, ADP_ERR_INVALID_ARG);
        return page;
      };
      // Where the next unit's groups of 16 positions lie (pages of 16 positions and more: a group lies in one page),
      // and whether all its positions are attended.
      int pg[RG], ahead[RG];
      bool next_full = false;
      auto fetch_pages = [&](int ut) {
        if constexpr (!SMALL) {
#pragma unroll
          for (int g = 0; g < RG; ++g) ahead[g] = page_at(ut * UNIT + g * 16, 16);
        }
      };
      auto take_pages = [&](int ut) {
        next_full = !SMALL && (WIN ? seen.all(ut * UNIT, UNIT) : (ut + 1) * UNIT <= len);
        if constexpr (!SMALL) {
#pragma unroll
          for (int g = 0; g < RG; ++g) {
            pg[g] = ahead[g];
            next_full &= pg[g] >= 0;
          }
        }
      };
      auto load_k16 = [&](int g, int j, const uint8_t* p) {
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) {
          const uint4 w = ldg16(p + kc * 64);
          kr[g][j][kc * 4] = w.x, kr[g][j][kc * 4 + 1] = w.y, kr[g][j][kc * 4 + 2] = w.z, kr[g][j][kc * 4 + 3] = w.w;
        }
      };
      auto load_v16 = [&](int g, int j, const uint8_t* p) {
        if constexpr (VB >= 16) {
#pragma unroll
          for (int h = 0; h < VB / 16; ++h) {
            const uint4 w = ldg16(p + h * 128);
            vr[g][j][h * 4] = w.x, vr[g][j][h * 4 + 1] = w.y, vr[g][j][h * 4 + 2] = w.z, vr[g][j][h * 4 + 3] = w.w;
          }
        } else {
          const uint2 w = ldg8(p);
          vr[g][j][0] = w.x, vr[g][j][1] = w.y;
        }
      };
      const int k_lane = r8 * ROWB + l4 * 16, v_lane = 2 * l4 * ROWB + r8 * (VB >= 16 ? 16 : 8);
      uint32_t kmask = 0;  // bit 2 g + j: position row j of group g is attended (of a unit that is not full)
      auto load_k = [&](int ut) {
        if (next_full) {
#pragma unroll
          for (int g = 0; g < RG; ++g) {
            const int cell = (kvh << c.log2_page) + ((ut * UNIT + g * 16) & in_page);
            const uint8_t* p = c.k + (int64_t)pg[g] * c.page_bytes + (int64_t)cell * ROWB + k_lane;
            load_k16(g, 0, p);
            load_k16(g, 1, p + 8 * ROWB);
            if constexpr (Q8) {
              const int64_t at = (int64_t)pg[g] * c.scale_stride + cell + r8;
              ksc[g][0] = __ldg(c.k_scale + at), ksc[g][1] = __ldg(c.k_scale + at + 8);
              vsc[g][0] = __ldg(c.v_scale + at), vsc[g][1] = __ldg(c.v_scale + at + 8);
            }
          }
          return;
        }
        kmask = 0;
#pragma unroll
        for (int g = 0; g < RG; ++g) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int pos = ut * UNIT + g * 16 + r8 + 8 * j;
            const int page = SMALL ? page_at(pos, 1) : pg[g];
            ksc[g][j] = vsc[g][j] = 0.0f;
            if (page >= 0 && (WIN ? seen.sees(pos) : pos < len)) {
              const int cell = (kvh << c.log2_page) + (pos & in_page);
              kmask |= 1u << (2 * g + j);
              load_k16(g, j, c.k + (int64_t)page * c.page_bytes + (int64_t)cell * ROWB + l4 * 16);
              if constexpr (Q8) {
                ksc[g][j] = __ldg(c.k_scale + (int64_t)page * c.scale_stride + cell);
                vsc[g][j] = __ldg(c.v_scale + (int64_t)page * c.scale_stride + cell);
              }
            } else {
#pragma unroll
              for (int w = 0; w < KC * 4; ++w) kr[g][j][w] = 0;
            }
          }
        }
      };
      auto load_v = [&](int ut, bool full) {
        if (full) {
#pragma unroll
          for (int g = 0; g < RG; ++g) {
            const int cell = (kvh << c.log2_page) + ((ut * UNIT + g * 16) & in_page);
            const uint8_t* p = c.v + (int64_t)pg[g] * c.page_bytes + (int64_t)cell * ROWB + v_lane;
#pragma unroll
            for (int j = 0; j < 4; ++j) load_v16(g, j, p + ((j & 1) + 8 * (j >> 1)) * ROWB);
          }
          return;
        }
#pragma unroll
        for (int g = 0; g < RG; ++g) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int pos = ut * UNIT + g * 16 + 2 * l4 + (j & 1) + 8 * (j >> 1);
            const int page = SMALL ? page_at(pos, 1) : pg[g];
            if (page >= 0 && (WIN ? seen.sees(pos) : pos < len)) {
              const int cell = (kvh << c.log2_page) + (pos & in_page);
              load_v16(g, j, c.v + (int64_t)page * c.page_bytes + (int64_t)cell * ROWB + r8 * (VB >= 16 ? 16 : 8));
            } else {
#pragma unroll
              for (int w = 0; w < VW; ++w) vr[g][j][w] = 0;
            }
          }
        }
      };

      auto unit = [&](int i) { return WIN ? seen.unit(i) : i; };
      fetch_pages(unit(t));
      take_pages(unit(t));
      if (n > 1) fetch_pages(unit(t + 1));
      load_k(unit(t));
      load_v(unit(t), next_full);
      for (int i = 0; i < n; ++i) {
        const bool more = i + 1 < n, full = next_full;
        if (more) {
          take_pages(unit(t + i + 1));
          if (i + 2 < n) fetch_pages(unit(t + i + 2));
        }
        // ---- S^T = K Q^T: rows are keys, columns heads
        float s[RG][NT][4];
#pragma unroll
        for (int g = 0; g < RG; ++g) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[g][nt][0] = s[g][nt][1] = s[g][nt][2] = s[g][nt][3] = 0.0f;
#pragma unroll
          for (int ks = 0; ks < MT; ++ks) {
            uint32_t f[4];
            if constexpr (Q8) {
              e4m3x4_to_f16(kr[g][0][ks], f[0], f[2]);
              e4m3x4_to_f16(kr[g][1][ks], f[1], f[3]);
            } else {
              f[0] = kr[g][0][2 * ks], f[1] = kr[g][1][2 * ks], f[2] = kr[g][0][2 * ks + 1], f[3] = kr[g][1][2 * ks + 1];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16<BF>(s[g][nt], f[0], f[1], f[2], f[3], qf[nt][ks][0], qf[nt][ks][1]);
          }
        }
        const uint32_t on = kmask;
        float ks_now[RG][2], vs_now[RG][2];
        if constexpr (Q8) {
#pragma unroll
          for (int g = 0; g < RG; ++g)
#pragma unroll
            for (int j = 0; j < 2; ++j) ks_now[g][j] = ksc[g][j], vs_now[g][j] = vsc[g][j];
        }
        if (more) load_k(unit(t + i + 1));
        // ---- scores in base-2 exponents; the running maxima are replaced only when some score (or e4m3's score + log2 of
        // the value scale, taken for the lane's largest score with its largest scale) exceeds its maximum by more than 8,
        // decided per warp: till then the weights stay below 2^8, and the same stale maximum scales O and l alike
        bool need = false;
        auto log2_scale = [](float s) { return fmaxf(log2_fast(fabsf(s)), -126.0f); };  // (2^-126: the least one)
        float lvtop = 0.0f;
        if constexpr (Q8) {
          float vtop = 0.0f;
#pragma unroll
          for (int g = 0; g < RG; ++g) vtop = fmaxf(vtop, fmaxf(fabsf(vs_now[g][0]), fabsf(vs_now[g][1])));
          lvtop = log2_scale(vtop);
        }
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            top[nt][j] = -INFINITY;
#pragma unroll
            for (int g = 0; g < RG; ++g)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                float x = s[g][nt][2 * r + j] * qs[nt][j];
                if constexpr (Q8) x *= ks_now[g][r];
                if (!full) x = (on >> (2 * g + r)) & 1 ? x : -INFINITY;
                s[g][nt][2 * r + j] = x;
                top[nt][j] = fmaxf(top[nt][j], x);
              }
            need |= top[nt][j] > m[nt][j] + kStale;
            if constexpr (Q8) need |= top[nt][j] + lvtop > mo[nt][j] + kStale;
          }
        }
        if (__any_sync(0xFFFFFFFFu, need)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float mn = top[nt][j];
#pragma unroll
              for (int d = 4; d <= 16; d <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, d));
              mn = fmaxf(m[nt][j], mn);
              float f = exp2_fast(m[nt][j] - safe_max(mn));
              m[nt][j] = mn;
              l[nt][j] *= f;
              if constexpr (Q8) {  // (both maxima at once: mo is m - 126 at least, and vc finite)
                float mw = -INFINITY;
#pragma unroll
                for (int g = 0; g < RG; ++g)
#pragma unroll
                  for (int r = 0; r < 2; ++r) mw = fmaxf(mw, s[g][nt][2 * r + j] + log2_scale(vs_now[g][r]));
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) mw = fmaxf(mw, __shfl_xor_sync(0xFFFFFFFFu, mw, d));
                mw = fmaxf(mo[nt][j], mw);
                f = exp2_fast(mo[nt][j] - safe_max(mw));
                mo[nt][j] = mw;
                vc[nt][j] = mw == -INFINITY ? 1.0f : exp2_fast(mn - mw);
              }
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                o[mt][nt][j] *= f;
                o[mt][nt][2 + j] *= f;
              }
            }
        }
        // ---- P, and O^T += V^T P^T
#pragma unroll
        for (int g = 0; g < RG; ++g) {
          // bf16's 8 bits would leave the weights' rounding as large as the result's: their remainder is weighed too
          // (error against 64 bits of one 131,011-position bf16 row: 2.6e-3 without, the plain form's 1.6e-3 with it)
          uint32_t pf[NT][2], pl[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float p0 = exp2_fast(s[g][nt][2 * r] - (safe_max(m[nt][0]) - kWeightUp<CDT>));
              float p1 = exp2_fast(s[g][nt][2 * r + 1] - (safe_max(m[nt][1]) - kWeightUp<CDT>));
              l[nt][0] += p0;
              l[nt][1] += p1;
              if constexpr (Q8) {  // (cut where the weight is 0 next to it, or as good as: 0 times infinity is none)
                p0 *= min_nan(vs_now[g][r] * vc[nt][0], kFactorMax);
                p1 *= min_nan(vs_now[g][r] * vc[nt][1], kFactorMax);
              }
              const uint32_t hi = pack2(p0, p1, BF ? DT_BF16 : DT_F16);
              pf[nt][r] = transpose8x8(hi);
              if constexpr (BF)
                pl[nt][r] = transpose8x8(pack2(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xFFFF0000u), DT_BF16));
            }
          }
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            const uint32_t x0 = vr[g][0][w], x1 = vr[g][1][w], x2 = vr[g][2][w], x3 = vr[g][3][w];
            if constexpr (Q8) {
              uint32_t f[8];
              e4m3x4_to_f16(__byte_perm(x0, x1, 0x5140), f[0], f[1]);
              e4m3x4_to_f16(__byte_perm(x2, x3, 0x5140), f[2], f[3]);
              e4m3x4_to_f16(__byte_perm(x0, x1, 0x7362), f[4], f[5]);
              e4m3x4_to_f16(__byte_perm(x2, x3, 0x7362), f[6], f[7]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16<BF>(o[2 * w][nt], f[0], f[1], f[2], f[3], pf[nt][0], pf[nt][1]);
                mma16<BF>(o[2 * w + 1][nt], f[4], f[5], f[6], f[7], pf[nt][0], pf[nt][1]);
              }
            } else {
              const uint32_t f0 = __byte_perm(x0, x1, 0x5410), f1 = __byte_perm(x0, x1, 0x7632);
              const uint32_t f2 = __byte_perm(x2, x3, 0x5410), f3 = __byte_perm(x2, x3, 0x7632);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16<BF>(o[w][nt], f0, f1, f2, f3, pf[nt][0], pf[nt][1]);
                if constexpr (BF) mma16<BF>(o[w][nt], f0, f1, f2, f3, pl[nt][0], pl[nt][1]);
              }
            }
          }
        }
        if (more) load_v(unit(t + i + 1), next_full);
      }

      // ---- end of the piece: sums over the lanes that share a head
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) l[nt][j] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][j], d);
      if constexpr (Q8) {  // O relative to m (in two steps, so that the factor does not leave fp32's range)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float f = mo[nt][j] == -INFINITY ? 0.0f : exp2_fast(0.5f * (mo[nt][j] - m[nt][j]));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              o[mt][nt][j] = o[mt][nt][j] * f * f;
              o[mt][nt][2 + j] = o[mt][nt][2 + j] * f * f;
            }
          }
      }
      // Element d of this lane's head 2 l4 + j: tile mt, register j (even d) and 2 + j (odd d).
      auto elem = [&](int mt) { return Q8 ? r8 * VB + 2 * mt : ((mt / 4) * 8 + r8) * 8 + 2 * (mt % 4); };
      const bool whole = t == 0 && n == n_units;
      if (whole) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int h = nt * 8 + 2 * l4 + j;
            if (h >= heads) continue;
            const float inv = l[nt][j] == 0.0f ? 0.0f : 1.0f / l[nt][j];
            uint8_t* po = a.out + (int64_t)b * a.out_stride + (int64_t)(kvh * a.group + head0 + h) * HD * 2;
#pragma unroll
            for (int mt = 0; mt < MT; mt += 4) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) w[e] = pack2(o[mt + e][nt][j] * inv, o[mt + e][nt][2 + j] * inv, QDT);
              *reinterpret_cast<uint4*>(po + elem(mt) * 2) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
      } else {
        const int sl = warp * 2 + (u == u_first ? 0 : 1);
        Part& P = slots[sl];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int h = nt * 8 + 2 * l4 + j;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              *reinterpret_cast<float2*>(&P.o[h][elem(mt)]) = make_float2(o[mt][nt][j], o[mt][nt][2 + j]);
            if (r8 == 0) {
              P.m[h] = m[nt][j];
              P.l[h] = l[nt][j];
            }
          }
        if (lane == 0) {
          s_seg[sl] = b * nvt + vt;
          s_u0[sl] = u - t;
          s_u1[sl] = u - t + n_units;
        }
      }
      u += n;
      t = 0;
      if (u < u_end && ++vt == nvt) {  // (never in a cluster: its warps' units are of one segment)
        vt = 0;
        do {
          ++b;
        } while (b < c.n_seqs && units_of(b) == 0);
        if (b >= c.n_seqs) break;
      }
    }
  }
  if (a.cluster) {
    // ---- join each CTA's pieces, then the cluster's; every CTA takes a part of the output
    __syncthreads();
    if (seg_units != 1) {  // (a single unit was written by its warp)
      const int kvh = vt0 / a.tiles, head0 = (vt0 % a.tiles) * (NT * 8);
      const int heads = min(NT * 8, a.group - head0), rank = blockIdx.x % a.cluster;
      for (int x = threadIdx.x; x < heads * (HD / 4); x += kPagedWarps * 32) {
        const int h = x / (HD / 4), d = (x % (HD / 4)) * 4;
        float m = -INFINITY, sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kPagedWarps; ++w)
          if (s_seg[w * 2] >= 0) m = fmaxf(m, slots[w * 2].m[h]);
#pragma unroll
        for (int w = 0; w < kPagedWarps; ++w) {
          if (s_seg[w * 2] < 0) continue;
          const float4 p = *reinterpret_cast<const float4*>(&slots[w * 2].o[h][d]);
          const float f = exp2_fast(slots[w * 2].m[h] - safe_max(m));
          sum = fmaf(f, slots[w * 2].l[h], sum);
          acc.x = fmaf(f, p.x, acc.x), acc.y = fmaf(f, p.y, acc.y), acc.z = fmaf(f, p.z, acc.z), acc.w = fmaf(f, p.w, acc.w);
        }
        // (into slots that no warp of a cluster uses)
        *reinterpret_cast<float4*>(&slots[1].o[h][d]) = acc;
        if (d == 0) slots[1].m[h] = m, slots[1].l[h] = sum;
      }
      cluster_barrier();
      for (int x = rank * kPagedWarps * 32 + threadIdx.x; x < heads * (HD / 4); x += a.cluster * kPagedWarps * 32) {
        const int h = x / (HD / 4), d = (x % (HD / 4)) * 4;
        float pm[8], pl[8];
        float4 po[8];
        float m = -INFINITY, sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          pm[k] = -INFINITY;
          if (k >= a.cluster) continue;
          const uint32_t at = cluster_addr(&slots[1], k);
          pm[k] = cluster_ld(at + (uint32_t)offsetof(Part, m) + 4 * h);
          pl[k] = cluster_ld(at + (uint32_t)offsetof(Part, l) + 4 * h);
          po[k] = cluster_ld4(at + (uint32_t)(h * HD + d) * 4);
          m = fmaxf(m, pm[k]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k >= a.cluster) continue;
          const float f = exp2_fast(pm[k] - safe_max(m));
          sum = fmaf(f, pl[k], sum);
          acc.x = fmaf(f, po[k].x, acc.x), acc.y = fmaf(f, po[k].y, acc.y);
          acc.z = fmaf(f, po[k].z, acc.z), acc.w = fmaf(f, po[k].w, acc.w);
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint8_t* dst = a.out + (int64_t)b0 * a.out_stride + ((int64_t)(kvh * a.group + head0 + h) * HD + d) * 2;
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack2(acc.x * inv, acc.y * inv, QDT), pack2(acc.z * inv, acc.w * inv, QDT));
      }
    } else {
      cluster_barrier();
    }
    cluster_barrier();  // no CTA leaves while another reads its shared memory
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();

  // ---- join the warps' pieces: consecutive slots of one segment
  if (threadIdx.x == 0) a.meta[blockIdx.x].seg = -1;
  for (int i = 0; i < kPagedWarps * 2;) {
    const int seg = s_seg[i];
    if (seg < 0) {
      ++i;
      continue;
    }
    int e = i + 1;
    while (e < kPagedWarps * 2 && (s_seg[e] < 0 || s_seg[e] == seg)) ++e;
    const int vt = seg % nvt, b = seg / nvt;
    const int kvh = vt / a.tiles, head0 = (vt % a.tiles) * (NT * 8);
    const int heads = min(NT * 8, a.group - head0);
    const bool before = s_u0[i] < c0, behind = s_u1[i] > c1;
    Part* dst = reinterpret_cast<Part*>(a.partials) + blockIdx.x * 2 + (before ? 0 : 1);
    for (int x = threadIdx.x; x < heads * (HD / 4); x += kPagedWarps * 32) {
      const int h = x / (HD / 4), d = (x % (HD / 4)) * 4;
      float top = -INFINITY;
      for (int k = i; k < e; ++k)
        if (s_seg[k] >= 0) top = fmaxf(top, slots[k].m[h]);
      float sum = 0.0f;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int k = i; k < e; ++k) {
        if (s_seg[k] < 0) continue;
        const float f = exp2_fast(slots[k].m[h] - safe_max(top));
        const float4 p = *reinterpret_cast<const float4*>(&slots[k].o[h][d]);
        sum = fmaf(f, slots[k].l[h], sum);
        acc.x = fmaf(f, p.x, acc.x), acc.y = fmaf(f, p.y, acc.y), acc.z = fmaf(f, p.z, acc.z), acc.w = fmaf(f, p.w, acc.w);
      }
      if (before || behind) {
        *reinterpret_cast<float4*>(&dst->o[h][d]) = acc;
        if (d == 0) dst->m[h] = top, dst->l[h] = sum;
      } else {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint8_t* po = a.out + (int64_t)b * a.out_stride + ((int64_t)(kvh * a.group + head0 + h) * HD + d) * 2;
        *reinterpret_cast<uint2*>(po) = make_uint2(pack2(acc.x * inv, acc.y * inv, QDT), pack2(acc.z * inv, acc.w * inv, QDT));
      }
    }
    if (!before && behind && threadIdx.x == 0) {
      a.meta[blockIdx.x].seg = seg;
      a.meta[blockIdx.x].last = split_owner(total, parts, s_u1[i] - 1);
    }
    i = e;
  }
}

// Joins the segments that several CTAs share: block (c, h) takes the segment that starts in CTA c and goes on behind
// it, and its head h.  JW warps read the parts in turn; the first threads join the warps' results.
template <int HD, int QDT, int NT, int JW>
__global__ void __launch_bounds__(JW * 32) paged_attention_join_kernel(AttnArgs a) {
  using Part = Partial<HD, NT>;
  constexpr int W = HD / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const SplitMeta meta = a.meta[blockIdx.x];
  if (meta.seg < 0) return;
  const int nvt = a.c.n_kv_heads * a.tiles;
  const int vt = meta.seg % nvt, b = meta.seg / nvt;
  const int kvh = vt / a.tiles, head0 = (vt % a.tiles) * (NT * 8), h = blockIdx.y;
  if (h >= min(NT * 8, a.group - head0)) return;
  const Part* parts = reinterpret_cast<const Part*>(a.partials);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = meta.last - (int)blockIdx.x + 1;
  // part 0 is this CTA's second slot, part k the first slot of CTA c + k
  float m = -INFINITY, l = 0.0f, o[W];
#pragma unroll
  for (int e = 0; e < W; ++e) o[e] = 0.0f;
#pragma unroll JW
  for (int k = warp; k < n; k += JW) {
    const Part& p = parts[(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)];
    const float pm = p.m[h], pl = p.l[h];
    float x[W];
#pragma unroll
    for (int e = 0; e < W; ++e) x[e] = p.o[h][e * 32 + lane];
    const float mn = fmaxf(m, pm);
    const float f = exp2_fast(m - safe_max(mn)), g = exp2_fast(pm - safe_max(mn));
    m = mn;
    l = fmaf(l, f, g * pl);
#pragma unroll
    for (int e = 0; e < W; ++e) o[e] = fmaf(o[e], f, g * x[e]);
  }
  __shared__ float s_m[JW], s_l[JW], s_o[JW][HD];
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
  for (int e = 0; e < W; ++e) s_o[warp][e * 32 + lane] = o[e];
  __syncthreads();
  float top = s_m[0];
#pragma unroll
  for (int w = 1; w < JW; ++w) top = fmaxf(top, s_m[w]);
  float sum = 0.0f, f[JW];
#pragma unroll
  for (int w = 0; w < JW; ++w) {
    f[w] = exp2_fast(s_m[w] - safe_max(top));
    sum = fmaf(f[w], s_l[w], sum);
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (threadIdx.x < HD / 2) {
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      x[e] = 0.0f;
#pragma unroll
      for (int w = 0; w < JW; ++w) x[e] = fmaf(f[w], s_o[w][threadIdx.x * 2 + e], x[e]);
    }
    uint8_t* po = a.out + (int64_t)b * a.out_stride + (int64_t)(kvh * a.group + head0 + h) * HD * 2;
    reinterpret_cast<uint32_t*>(po)[threadIdx.x] = pack2(x[0] * inv, x[1] * inv, QDT);
  }
}

// ---------------------------------------------------------------- host side

// Query heads per KV head take tiles of 8 (a group of up to 8) or 16 columns of the tensor instruction (16: K and V are
// read once for up to 16 heads, where tiles of 8 would read them twice).
inline int head_tiles(int group) { return group <= 8 ? 1 : 2; }

// How an attention call falls on the GPU: a cluster of CTAs per segment, or CTAs that share all units evenly.
struct AttentionPlan {
  int nt, tiles, cluster, ctas;
  size_t bytes;  // workspace
};

// A cluster per segment while all of them can be resident and no warp gets more than kClusterUnits units even if every
// sequence fills its table: then the uneven lengths cost less than the even split's sums, partial results and second
// launch.  (Clusters take up to 8 CTAs, the portable size, and no more warps than there are units.)
// Cluster and even split, us on the GPU: 1 x 77 positions of 4 KV heads 4.7 and 8.8; 4 x 1,024 of 4 7.3 and 10.8; 4 x 4,096
// of 8 (8 units a warp) 14.7 and 17.6; 57 x 500 of 8 18.5 and 21.0; the worst, 14 x 1,000 of 8, 17.8 and 16.3.
constexpr int kClusterUnits = 8;

// Units of a sequence that fills its table, or its window and first positions (window 0: none; both may start inside a unit).
inline int64_t full_units(const adp_paged_kv* kv, int32_t window, int32_t sinks) {
  const int unit = 4096 / (kv->head_dim * elem_bytes(kv->dtype));
  const int64_t all = ((int64_t)kv->table_width * kv->page_size + unit - 1) / unit;
  const int64_t seen = ((int64_t)window + unit - 1) / unit + 1 + ((int64_t)sinks + unit - 1) / unit;
  return window && seen < all ? seen : all;
}

inline AttentionPlan attention_plan(const adp_paged_kv* kv, int group, int sms, int32_t window, int32_t sinks) {
  AttentionPlan p{};
  p.nt = head_tiles(group);
  p.tiles = (group + p.nt * 8 - 1) / (p.nt * 8);
  const int resident = sms * (p.nt == 1 ? kResident<1> : kResident<2>);
  const int64_t per_seq = full_units(kv, window, sinks);
  const int64_t segs = (int64_t)kv->n_seqs * kv->n_kv_heads * p.tiles;
  if (segs > 0 && segs <= resident) {
    int cs = 1;
    while (cs < 8 && segs * cs * 2 <= resident && cs * kPagedWarps < per_seq) cs *= 2;
    if (per_seq <= (int64_t)cs * kPagedWarps * kClusterUnits) {
      p.cluster = cs;
      p.ctas = (int)segs * cs;
      return p;
    }
  }
  p.ctas = split_parts(per_seq * (segs > 0 ? segs : 1), resident);
  p.bytes = (size_t)p.ctas * 2 * (p.nt * 8) * (kv->head_dim + 2) * sizeof(float) + (size_t)p.ctas * sizeof(SplitMeta);
  return p;
}

template <int HD, int CDT, int QDT, int NT, bool SMALL, bool WIN>
struct AttentionKey {};

template <int HD, int CDT, int QDT, int NT, bool SMALL, bool WIN>
cudaError_t attention_launch(const AttnArgs& a, int ctas, cudaStream_t st) {
  constexpr size_t smem = sizeof(Partial<HD, NT>) * kPagedWarps * 2;
  auto* kernel = paged_attention_kernel<HD, CDT, QDT, NT, SMALL, WIN>;
  cudaError_t e = allow_smem<AttentionKey<HD, CDT, QDT, NT, SMALL, WIN>>((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  if (a.cluster > 1) {
    cudaLaunchAttribute together{};
    together.id = cudaLaunchAttributeClusterDimension;
    together.val.clusterDim.x = a.cluster;
    together.val.clusterDim.y = together.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPagedWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &together;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
  }
  kernel<<<ctas, kPagedWarps * 32, smem, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.cluster || ctas == 1) return e;  // one CTA shares no segment
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas - 1, a.group < NT * 8 ? a.group : NT * 8);  // no segment goes on behind the last CTA
  // (one long context is cut into many parts, and a window leaves little else to wait for: 131,011 positions behind a window of
  // 32,768)
  constexpr int kJoinWarps = WIN ? 8 : 4;
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_attention_join_kernel<HD, QDT, NT, kJoinWarps>, a);
}

inline int attention_check(const adp_paged_kv* kv, int32_t n_heads, PagedView* c) {
  const int rc = paged_view(kv, c);
  if (rc) return rc;
  if (n_heads < 1 || n_heads % kv->n_kv_heads) return ADP_ERR_INVALID_ARG;
  if (n_heads > 4096 || kv->n_seqs > kPagedMaxSeqs) return ADP_ERR_UNSUPPORTED_CONFIG;
  // (the units of 32 sequences are added in 32 bits)
  if ((kv->n_seqs < 32 ? kv->n_seqs : 32) * full_units(kv, 0, 0) > 0x7FFFFFFF) return ADP_ERR_UNSUPPORTED_CONFIG;
  return ADP_OK;
}

inline int attention_workspace(const adp_paged_kv* kv, int32_t n_heads, int32_t window, int32_t sinks, uint64_t* bytes) {
  PagedView c;
  int rc = bytes ? attention_check(kv, n_heads, &c) : ADP_ERR_INVALID_ARG;
  int sms = 0;
  if (rc || (rc = sm_count(&sms))) return rc;
  const int group = n_heads / kv->n_kv_heads;
  *bytes = attention_plan(kv, group, sms, window, sinks).bytes;
  return ADP_OK;
}

template <bool WIN>
int attention_run(const adp_paged_kv* kv, const void* q, int32_t q_dtype, int32_t n_heads, int64_t q_stride, float scale,
                  int32_t window, int32_t sinks, void* out, int64_t out_stride, void* workspace, uint64_t workspace_bytes,
                  int32_t* dev_status, void* cuda_stream, const char* where) {
  AttnArgs a{};
  int rc = attention_check(kv, n_heads, &a.c);
  if (rc) return rc;
  if (q_dtype != ADP_F16 && q_dtype != ADP_BF16) return ADP_ERR_UNSUPPORTED_CONFIG;
  if (kv->dtype != ADP_E4M3 && kv->dtype != q_dtype) return ADP_ERR_UNSUPPORTED_CONFIG;
  const int64_t width = (int64_t)n_heads * kv->head_dim;
  if (!isfinite(scale) || ((uintptr_t)dev_status & 3)) return ADP_ERR_INVALID_ARG;
  if (kv->n_seqs == 0) return ADP_OK;
  if (!q || !out || !aligned16(q) || !aligned16(out) || q_stride < width || out_stride < width || q_stride % 8 || out_stride % 8)
    return ADP_ERR_INVALID_ARG;
  int sms = 0;
  if ((rc = sm_count(&sms))) return rc;
  const int group = n_heads / kv->n_kv_heads;
  const AttentionPlan plan = attention_plan(kv, group, sms, window, sinks);
  const int nt = plan.nt, ctas = plan.ctas;
  if (plan.bytes && (!workspace || !aligned16(workspace) || workspace_bytes < plan.bytes)) return ADP_ERR_INVALID_ARG;
  a.q = static_cast<const uint8_t*>(q);
  a.out = static_cast<uint8_t*>(out);
  a.q_stride = q_stride * 2;
  a.out_stride = out_stride * 2;
  a.group = group;
  a.tiles = plan.tiles;
  a.cluster = plan.cluster;
  a.window = window;
  a.sinks = sinks;
  a.scale_log2 = log2_scale(scale);
  if (plan.bytes) {
    a.partials = workspace;
    a.meta = reinterpret_cast<SplitMeta*>(static_cast<uint8_t*>(workspace) + plan.bytes - (size_t)ctas * sizeof(SplitMeta));
  }
  a.status = dev_status;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const bool small = kv->page_size < 16;
  cudaError_t e = cudaErrorInvalidValue;
  auto by_page = [&](auto hd, auto cdt, auto qdt, auto n) {
    constexpr int H = decltype(hd)::value, C = decltype(cdt)::value, Q = decltype(qdt)::value, N = decltype(n)::value;
    e = small ? attention_launch<H, C, Q, N, true, WIN>(a, ctas, st) : attention_launch<H, C, Q, N, false, WIN>(a, ctas, st);
  };
  auto by_group = [&](auto hd, auto cdt, auto qdt) {
    if (nt == 1) by_page(hd, cdt, qdt, std::integral_constant<int, 1>());
    else by_page(hd, cdt, qdt, std::integral_constant<int, 2>());
  };
  auto by_type = [&](auto hd) {
    using F = std::integral_constant<int, DT_F16>;
    using B = std::integral_constant<int, DT_BF16>;
    using E = std::integral_constant<int, DT_E4M3>;
    if (kv->dtype == ADP_F16) by_group(hd, F(), F());
    else if (kv->dtype == ADP_BF16) by_group(hd, B(), B());
    else if (q_dtype == ADP_F16) by_group(hd, E(), F());
    else by_group(hd, E(), B());
  };
  if (kv->head_dim == 128) by_type(std::integral_constant<int, 128>());
  else by_type(std::integral_constant<int, 64>());
  return cuda_status(e, where);
}

}  // namespace
}  // namespace adp
