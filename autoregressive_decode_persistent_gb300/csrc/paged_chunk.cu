// Attention of every sequence's last rows over the pages of a KV cache, on the tensor cores.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "../../include/adp.h"
#include "device.cuh"
#include "paged.cuh"
#include "paged_chunk.h"
#include "tc.cuh"
#include "tc_attention.cuh"

namespace adp {
namespace {

constexpr int kRows = 128;              // rows of a query tile (M of the MMA)
constexpr int kKeys = kChunkKeys;
constexpr float kRescale = 8.0f;        // base-2 growth of a row's maximum that rescales its output
constexpr float kFactorMax = 1.329227996e36f;  // 2^120, of a value scale relative to the largest product
constexpr int kItems = 2;               // the piece of work and the next one

// What a CTA has left for the join: its first piece's first part may go on from the CTA before, its last one may go on behind it.
struct ChunkMeta {
  int32_t first;              // slot 0: 0 unused, 1 a part that goes on behind this CTA, 2 the last part of its piece
  int32_t starts;             // slot 1 holds the first part of a piece
  int32_t row0, tokens, head;  // that piece: its first packed row, tokens, KV head
  int32_t pad[3];
};

struct ChunkArgs {
  PagedView c;
  const int32_t* cu;
  uint8_t* out;
  int64_t out_stride;            // bytes
  int32_t n_rows, group, tok;    // query heads per KV head; tokens of a tile
  int32_t window, sinks;
  float scale_log2;              // of |scale|, and above 0
  uint32_t neg;                  // scale < 0: the instruction descriptor's bit that negates A
  int32_t rows_cap;              // rows of a partial result (128 or 256)
  float* part_o;                 // [ctas][2][rows_cap][head_dim]
  float2* part_ml;               // [ctas][2][rows_cap]
  ChunkMeta* meta;               // [ctas]
  int32_t* status;
  uint64_t wait_ns;
};

// A sequence's new rows, within the packed rows, and its length, within its table.
struct Rows {
  int32_t q0, lq, len;
};
__device__ __forceinline__ Rows rows_of(const ChunkArgs& a, int b, int32_t* status) {
  Rows r;
  packed_range(a.cu, b, a.n_rows, status, &r.q0, &r.lq);
  const int32_t raw = a.c.lens[b];
  r.len = paged_length(raw, a.c.table_width, a.c.log2_page);
  if (raw > r.len) report(status, ADP_ERR_CONTEXT_OVERFLOW);
  if (raw < r.len || r.lq > r.len || (b == 0 && a.cu[0] != 0)) report(status, ADP_ERR_INVALID_ARG);
  return r;
}

// One piece of work: up to 2 x tok tokens from t0 on of a sequence for one KV head's group of query heads, and blocks
// [i0, i1) of the line that they see.
struct Item {
  int32_t q0, lq, len, b, t0, h;
  int32_t i0, i1;
  int32_t part;  // -1: all of its blocks; else the slot of the partial result
  int32_t stop;  // no work is left
  __device__ __forceinline__ int first() const { return len - lq + t0; }
  __device__ __forceinline__ int last(int span) const { return len - lq + min(t0 + span, lq) - 1; }
  // its rows fit one tile: the tiles are two halves of the blocks, in turn
  __device__ __forceinline__ bool half(int tok) const { return lq - t0 <= tok; }
};
// Blocks that tile t of the item works on, and the way from one to the next.
struct Own {
  int n, step, off;
};
__device__ __forceinline__ Own own_blocks(const Item& w, const ChunkSpan& s, int t, int tok) {
  const int n = w.i1 - w.i0;
  if (w.half(tok)) return Own{(n + 1 - t) / 2, 2, t};
  if (t == 1) return Own{n, 1, 0};
  const int last = w.first() + tok - 1;  // what tile A's last row sees is a beginning of the line
  return Own{last < 0 ? 0 : min(max(last / kKeys + 1 - s.gap - w.i0, 0), n), 1, 0};
}
// Whether some row of the item does not see all positions of the block at position kb.
__device__ __forceinline__ bool edge_block(int kb, int first, int last, int window, int sinks) {
  return kb + kKeys - 1 > first || (kb <= last - window && kb + kKeys - 1 >= sinks);
}

// The line of all work: sequences, in them pairs of tiles of tokens, in them KV heads, in them blocks.
struct Place {
  int32_t b, t, h, j;  // sequence, pair, KV head, block; b = n_seqs: the end
};

__device__ __forceinline__ int pair_blocks(const ChunkArgs& a, const Rows& r, int t) {
  const int span = 2 * a.tok, first = r.len - r.lq + t * span, last = r.len - r.lq + min((t + 1) * span, r.lq) - 1;
  return chunk_span(first, last, a.window, a.sinks).n;
}
// Units of a sequence for one KV head, one lane per sequence; long ones are added up by the whole warp.
__device__ __forceinline__ int64_t sequence_units(const ChunkArgs& a, const Rows& r, int lane) {
  constexpr int kAlone = 4;
  const int span = 2 * a.tok, pairs = (r.lq + span - 1) / span;
  int64_t sum = 0;
  if (pairs <= kAlone)
    for (int t = 0; t < pairs; ++t) sum += pair_blocks(a, r, t) + kChunkOver;
  for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, pairs > kAlone); todo; todo &= todo - 1) {
    const int l = __ffs(todo) - 1;
    const Rows o{__shfl_sync(0xFFFFFFFFu, r.q0, l), __shfl_sync(0xFFFFFFFFu, r.lq, l), __shfl_sync(0xFFFFFFFFu, r.len, l)};
    const int n = __shfl_sync(0xFFFFFFFFu, pairs, l);
    int64_t s = 0;
    for (int t = lane; t < n; t += 32) s += pair_blocks(a, o, t) + kChunkOver;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    if (lane == l) sum = s;
  }
  return sum;
}
__device__ __forceinline__ int64_t scan_inclusive(int64_t x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += o;
  }
  return x;
}
// Where a cut of the line at unit x goes.  chunks: units in front of every 32 sequences, for one KV head.  A whole warp asks.
__device__ __noinline__ Place find_place(const ChunkArgs& a, const int64_t* chunks, int n_chunks, int64_t x, int lane) {
  const int hkv = a.c.n_kv_heads;
  if (x >= chunks[n_chunks] * hkv) return Place{a.c.n_seqs, 0, 0, 0};
  int ch = 0;
  for (int at = 0; at < n_chunks; at += 32) {
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, at + lane < n_chunks && chunks[at + lane] * hkv <= x));
    if (n) ch = at + n - 1;
    if (n < 32) break;
  }
  x -= chunks[ch] * hkv;
  Rows r{0, 0, 0};
  if (ch * 32 + lane < a.c.n_seqs) r = rows_of(a, ch * 32 + lane, nullptr);
  const int64_t units = sequence_units(a, r, lane), upto = scan_inclusive(units, lane);
  const int l = min(__popc(__ballot_sync(0xFFFFFFFFu, upto * hkv <= x)), 31);
  x -= __shfl_sync(0xFFFFFFFFu, upto - units, l) * hkv;
  const Rows o{__shfl_sync(0xFFFFFFFFu, r.q0, l), __shfl_sync(0xFFFFFFFFu, r.lq, l), __shfl_sync(0xFFFFFFFFu, r.len, l)};
  const int span = 2 * a.tok, pairs = (o.lq + span - 1) / span;
  for (int t0 = 0; t0 < pairs; t0 += 32) {
    const int blocks = t0 + lane < pairs ? pair_blocks(a, o, t0 + lane) : 0;
    const int64_t mine = t0 + lane < pairs ? blocks + kChunkOver : 0, sum = scan_inclusive(mine, lane);
    const int p = __popc(__ballot_sync(0xFFFFFFFFu, sum * hkv <= x));
    if (p == 32) {
      x -= __shfl_sync(0xFFFFFFFFu, sum, 31) * hkv;
      continue;
    }
    x -= __shfl_sync(0xFFFFFFFFu, sum - mine, p) * hkv;
    const int n = __shfl_sync(0xFFFFFFFFu, blocks, p);
    const int h = (int)min(x / (n + kChunkOver), (int64_t)hkv - 1);
    return Place{ch * 32 + l, t0 + p, h, chunk_cut(n, x - (int64_t)h * (n + kChunkOver))};
  }
  return Place{a.c.n_seqs, 0, 0, 0};  // (the offsets changed while this call ran)
}

// Per ring slot of e4m3 blocks: the scales, log2 of the value scales and its largest over each half of the block.
struct SlotScales {
  float k[kKeys], v[kKeys], lv[kKeys], top[4];
};

template <int HD, int CDT>
struct ChunkSmem {
  static constexpr bool kConv = CDT == DT_E4M3;
  static constexpr int kSlots = kConv ? (HD == 128 ? 3 : 6) : (HD == 128 ? 5 : 8);  // of a block of K and one of V
  static constexpr int kRaw = kConv ? (HD == 128 ? 3 : 6) : 0;                       // blocks of codes under way
  static constexpr uint32_t kQBlock = 128 * 128;            // 128 rows x 64 elements, swizzled
  static constexpr uint32_t kQTile = (HD / 64) * kQBlock;
  static constexpr uint32_t kBlock = kKeys * 128;           // the same of K or V
  static constexpr uint32_t kTile = (HD / 64) * kBlock;
  static constexpr uint32_t kPair = 2 * kTile;
  static constexpr uint32_t kRawBytes = 2 * kKeys * HD + 512;  // codes, and a scale per row of K and V
  static constexpr uint32_t kRawAt = 2 * kQTile + kSlots * kPair;
  static constexpr uint32_t kScales = kRawAt + kRaw * kRawBytes;                           // [kSlots], e4m3
  static constexpr uint32_t kQf = kScales + (kConv ? kSlots * sizeof(SlotScales) : 0);     // [256] of the rows of Q, e4m3
  static constexpr uint32_t kHalf = kQf + (kConv ? 2 * kRows * 4 : 0);                     // [2 or 3][128]
  static constexpr uint32_t kCtl = kHalf + (kConv ? 3 : 2) * kRows * 4;
  static constexpr size_t kBytes = 1024 + kCtl + 512;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xFFFFu), __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
__device__ __forceinline__ float log2_scale_of(float s) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fabsf(s)));
  return fmaxf(y, -126.0f);  // (2^-126: the least scale there is)
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// CDT: the pages' type; QDT: the queries' (that of 16-bit pages).  LOAD: four warps bring K and V into the ring (e4m3 pages,
// which become fp16 there, and pages too small for tensor copies), else tensor copies do.
template <int HD, int CDT, int QDT, bool LOAD>
__global__ void __launch_bounds__(LOAD ? 512 : 384, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, const ChunkArgs a) {
  using L = ChunkSmem<HD, CDT>;
  constexpr int NS = L::kSlots;
  constexpr bool Q8 = CDT == DT_E4M3;
  constexpr bool BF = CDT == DT_BF16;               // the MMAs' type (e4m3: fp16)
  constexpr bool QCONV = Q8 && QDT == DT_BF16;      // bf16 queries beside fp16 codes
  static_assert(LOAD || !Q8, "");
  constexpr int kWarps = LOAD ? 16 : 12;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* Qs = smem;
  uint8_t* ring = smem + 2 * L::kQTile;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kCtl);
  uint64_t* full = bar;               // [NS]
  uint64_t* empty = full + NS;        // [NS]
  uint64_t* qfull = empty + NS;
  uint64_t* qready = qfull + 1;       // (QCONV)
  uint64_t* qempty = qready + 1;
  uint64_t* hfull = qempty + 1;       // tile B's half is done, and read
  uint64_t* hfree = hfull + 1;
  uint64_t* done = hfree + 1;
  uint64_t* sfull = done + 1;         // [2][2]: tile, buffer
  uint64_t* pready = sfull + 4;       // [2][2]
  uint64_t* odone = pready + 4;       // [2][2]
  uint64_t* ifull = odone + 4;        // [kItems]
  uint64_t* iempty = ifull + kItems;  // [kItems]
  uint64_t* hole = iempty + kItems;   // [NS]: positions of the block whose page has no place
  int32_t* ctl = reinterpret_cast<int32_t*>(hole + NS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctl);
  volatile int32_t* ab = ctl + 1;
  volatile int32_t* bad = ctl + 2;    // a non-finite value was taken out of an edge block
  volatile int32_t* holes = ctl + 3;  // some block had a position without a page
  Item* items = reinterpret_cast<Item*>(ctl + 6);  // [kItems]; the waits' limit lies in front
  float* s_half = reinterpret_cast<float*>(smem + L::kHalf);  // tile B's half of an item: maxima, sums, e4m3's factors of its output
  float* s_qf = reinterpret_cast<float*>(smem + L::kQf);
  SlotScales* s_scale = reinterpret_cast<SlotScales*>(smem + L::kScales);
  __shared__ Place s_cut[2];
  static_assert((2 * NS + 22) * 8 + NS * 8 + 24 + kItems * sizeof(Item) <= 512, "the control words' room");
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], LOAD ? 4 : 1);
      mbar_init(&empty[s], 2);  // tiles
      hole[s] = 0;
    }
    mbar_init(qfull, 1);
    mbar_init(qready, 8);
    mbar_init(qempty, 2);
    mbar_init(hfull, 4);
    mbar_init(hfree, 4);
    mbar_init(done, 2);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pready[i], 4);  // warps
      mbar_init(&odone[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&ifull[i], 1);
      mbar_init(&iempty[i], 10 + (LOAD ? 4 : 1));  // the issuing and the softmax warps, those that load
    }
    *ab = 0;
    *bad = 0;
    *holes = 0;
    *reinterpret_cast<uint64_t*>(ctl + 4) = a.wait_ns;
    mbar_fence_init();
  }
  // ---- the line of all work: units of every 32 sequences, their running sums, and this CTA's cuts
  const int n_chunks = (a.c.n_seqs + 31) / 32, span = 2 * a.tok;
  int64_t* chunks = reinterpret_cast<int64_t*>(smem);  // [n_chunks + 1], and a count (before anything is copied there)
  unsigned long long* s_items = reinterpret_cast<unsigned long long*>(chunks + n_chunks + 1);
  if (threadIdx.x == 0) *s_items = 0;
  __syncthreads();
  for (int ch = warp; ch < n_chunks; ch += kWarps) {
    Rows r{0, 0, 0};
    if (ch * 32 + lane < a.c.n_seqs) r = rows_of(a, ch * 32 + lane, a.status);
    int64_t n = sequence_units(a, r, lane);
    int pairs = (r.lq + span - 1) / span;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, d);
    pairs = __reduce_add_sync(0xFFFFFFFFu, pairs);
    if (lane == 0) {
      chunks[ch] = n;
      atomicAdd(s_items, (unsigned long long)pairs);
    }
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  if (warp == 0) {
    int64_t run = 0;
    for (int ch = 0; ch <= n_chunks; ch += 32) {
      const int64_t n = ch + lane < n_chunks ? chunks[ch + lane] : 0, sum = scan_inclusive(n, lane);
      if (ch + lane <= n_chunks) chunks[ch + lane] = run + sum - n;
      run += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
  }
  __syncthreads();
  const int64_t total = chunks[n_chunks] * a.c.n_kv_heads;
  const int parts = chunk_parts(total, (int64_t)*s_items * a.c.n_kv_heads, gridDim.x);
  if (warp < 2) {
    const int c = (int)blockIdx.x + warp;
    const Place p = find_place(a, chunks, n_chunks, c >= parts ? total : split_begin(total, parts, c), lane);
    if (lane == 0) s_cut[warp] = p;
  }
  fence_async_smem();  // (the sums have been read before copies take their place)
  __syncthreads();
  int32_t never = 0;

  if (warp >= 8 && warp < 12) {
    if (warp == 10) {
      // ---- finds the pieces of work of this CTA's range and asks for their queries
      Place p = s_cut[0];
      const Place end = s_cut[1];
      ChunkMeta left{};
      int published = 0, nq = 0;
      bool ok = true;
      Rows r{0, 0, 0};
      int pairs = 0;
      auto enter = [&]() {  // the sequence p.b
        if (p.b < a.c.n_seqs) r = rows_of(a, p.b, nullptr);
        else r = Rows{0, 0, 0};
        pairs = (r.lq + span - 1) / span;
      };
      auto before_end = [&]() {
        return p.b != end.b ? p.b < end.b : p.t != end.t ? p.t < end.t : p.h != end.h ? p.h < end.h : p.j < end.j;
      };
      enter();
      while (ok && p.b < a.c.n_seqs && before_end()) {
        if (p.t >= pairs) {  // the next sequence with rows
          p.t = p.h = p.j = 0;
          int b = p.b + 1;
          while (b < a.c.n_seqs) {
            const bool some = b + lane < a.c.n_seqs && rows_of(a, b + lane, nullptr).lq > 0;
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, some);
            if (m) {
              b += __ffs(m) - 1;
              break;
            }
            b += 32;
          }
          p.b = min(b, a.c.n_seqs);
          enter();
          continue;
        }
        const int n = pair_blocks(a, r, p.t);
        const bool here = p.b == end.b && p.t == end.t && p.h == end.h;
        const int i1 = here ? min(end.j, n) : n;
        if (p.j < i1 || n == 0) {
          const int s = published % kItems;
          if (published >= kItems && !(ok = mbar_wait_warp(&iempty[s], (published / kItems - 1) & 1, ab))) break;
          const bool before = p.j > 0, behind = i1 < n;
          const Item w{r.q0, r.lq, r.len, p.b, p.t * span, p.h, p.j, i1, before ? 0 : behind ? 1 : -1, 0};
          if (before) left.first = behind ? 1 : 2;
          if (!before && behind) {
            left.starts = 1;
            left.row0 = r.q0 + w.t0;
            left.tokens = min(span, r.lq - w.t0);
            left.head = p.h;
          }
          __syncwarp();
          if (lane == 0) {
            items[s] = w;
            mbar_arrive(&ifull[s]);
          }
          ++published;
          if (i1 > p.j) {
            if (nq > 0 && !(ok = mbar_wait_warp(qempty, (nq - 1) & 1, ab))) break;
            if (lane == 0) {
              const int tiles = w.half(a.tok) ? 1 : 2;
              mbar_arrive_expect_tx(qfull, (uint32_t)(tiles * a.tok * a.group) * 128 * (HD / 64));
              for (int t = 0; t < tiles; ++t)
                for (int c = 0; c < HD / 64; ++c)
                  tma_load_3d(Qs + t * L::kQTile + c * L::kQBlock, &mq, c * 64, w.h * a.group, w.q0 + w.t0 + t * a.tok, qfull);
            }
            ++nq;
            __syncwarp();
          }
        }
        p.j = 0;
        if (++p.h == a.c.n_kv_heads) p.h = 0, ++p.t;
      }
      if (ok) {
        const int s = published % kItems;
        ok = published < kItems || mbar_wait_warp(&iempty[s], (published / kItems - 1) & 1, ab);
        if (ok && lane == 0) {
          items[s].stop = 1;
          mbar_arrive(&ifull[s]);
        }
      }
      if (!ok) *ab = 1;
      if (lane == 0 && a.meta) a.meta[blockIdx.x] = left;
      // no copy may still be writing this CTA's shared memory when it exits
      if (nq > 0) mbar_wait(qfull, (nq - 1) & 1, &never, a.wait_ns);
      __syncwarp();
    } else if (warp == 8) {
      if constexpr (!LOAD) {
        // ---- copies blocks of K and V: a lane for every box of 64 elements x the rows of a page
        const int lg = min(a.c.log2_page, 6), box = 1 << lg, boxes = kKeys >> lg;
        const int bi = lane & (boxes - 1), kind = lane / boxes, col = kind % (HD / 64);
        const bool is_v = kind / (HD / 64) == 1, on = kind < 2 * (HD / 64);
        const uint32_t to = (uint32_t)(kind * L::kBlock + bi * box * 128);
        int g = 0;
        bool ok = true;
        uint32_t dirty = 0;  // slots whose positions without a page have been said
        for (int it = 0; ok; ++it) {
          const int is = it % kItems;
          if (!(ok = mbar_wait_warp(&ifull[is], (it / kItems) & 1, ab))) break;
          const Item w = items[is];
          __syncwarp();
          if (lane == 0) mbar_arrive(&iempty[is]);
          if (w.stop) break;
          const int last = w.last(span);
          const ChunkSpan sp = chunk_span(w.first(), last, a.window, a.sinks);
          const int32_t* trow = a.c.table + (int64_t)w.b * a.c.table_width;
          auto page_of = [&](int i) {  // of this lane's box: -2 where nothing of it is seen, -1 where it has no place
            const int pos = chunk_block(sp, i) * kKeys + bi * box;
            if (pos > last || (pos + box <= sp.low && pos >= a.sinks)) return -2;
            return paged_page(trow, a.c.table_width, a.c.n_pages, a.c.log2_page, pos);
          };
          int next = w.i0 < w.i1 ? page_of(w.i0) : -2;
          for (int i = w.i0; i < w.i1; ++i) {
            const int page = next, s = g % NS;
            if (i + 1 < w.i1) next = page_of(i + 1);
            if (g >= NS && !(ok = mbar_wait_warp(&empty[s], (g / NS - 1) & 1, ab))) break;
            const uint32_t out = __ballot_sync(0xFFFFFFFFu, page == -1) & (boxes == 32 ? ~0u : (1u << boxes) - 1);
            if (out || ((dirty >> s) & 1)) {
              if (lane == 0) {
                uint64_t m = 0;
                for (int k = 0; k < boxes; ++k)
                  if ((out >> k) & 1) m |= (box == 64 ? ~0ull : (1ull << box) - 1) << (k * box);
                hole[s] = m;
                if (out) {
                  *holes = 1;
                  report(a.status, ADP_ERR_INVALID_ARG);
                }
              }
              dirty = out ? dirty | (1u << s) : dirty & ~(1u << s);
            }
            if (lane == 0) mbar_arrive_expect_tx(&full[s], L::kPair);
            __syncwarp();
            if (on) {
              const int pos = chunk_block(sp, i) * kKeys + bi * box;
              // (a page number behind the pool: zeros)
              tma_load_4d(ring + s * L::kPair + to, is_v ? &mv : &mk, col * 64, pos & ((1 << a.c.log2_page) - 1), w.h,
                          page < 0 ? a.c.n_pages : page, &full[s]);
            }
            __syncwarp();
            ++g;
          }
        }
        if (!ok) *ab = 1;
        if (lane == 0)
          for (int i = g > NS ? g - NS : 0; i < g; ++i) mbar_wait(&full[i % NS], (i / NS) & 1, &never, a.wait_ns);
        __syncwarp();
      }
    } else {
      // ---- warps 9 and 11 issue the MMAs of tile A and of tile B, as the packed prompts' kernel has them
      constexpr uint32_t id_s0 = tc_idesc_f16(BF, 128, kKeys);
      constexpr uint32_t id_o = tc_idesc_f16(BF, 128, HD) | kTcIdescBMn;
      constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);
      const uint32_t id_s = id_s0 | a.neg;
      const uint32_t t = warp == 11;
      const uint32_t q_lo0 = (smem_u32(Qs) >> 4) | (1u << 16);
      const uint32_t k_lo = (smem_u32(ring) >> 4) | (1u << 16);
      const uint32_t v_lo = ((smem_u32(ring) + L::kTile) >> 4) | ((L::kBlock >> 4) << 16);
      const uint32_t tS = tmem + t * 128, tO = tmem + 256 + t * 128;
      uint32_t ks = 0, kphase = 0, vs = 0;  // the ring's next block, and the slot of the next own block to weigh
      uint32_t s_buf = 0, s_phase = 0, p_buf = 0, p_phase = 0, q_phase = 0;
      bool ok = true;
#pragma unroll 1
      for (int it = 0; ok; ++it) {
        const int is = it % kItems;
        if (!(ok = mbar_wait_warp(&ifull[is], (it / kItems) & 1, ab))) break;
        const Item w = items[is];
        __syncwarp();
        if (elect_one()) mbar_arrive(&iempty[is]);
        __syncwarp();
        if (w.stop) break;
        const int n = w.i1 - w.i0;
        if (n == 0) continue;
        const Own own = own_blocks(w, chunk_span(w.first(), w.last(span), a.window, a.sinks), t, a.tok);
        const uint32_t q_lo = q_lo0 + (w.half(a.tok) ? 0 : t * (L::kQTile >> 4));
        if (!(ok = mbar_wait_warp(QCONV ? qready : qfull, q_phase, ab))) break;
        q_phase ^= 1;
        int at = 0;  // blocks of the item that have been waited for
        vs = (ks + own.off) % NS;
        // the next block of the item, which is this tile's or not (then it is freed)
        auto skip = [&]() {
          if (!mbar_wait_warp(&full[ks], kphase, ab)) return false;
          if (elect_one()) mbar_arrive(&empty[ks]);
          __syncwarp();
          ++at;
          if (++ks == NS) ks = 0, kphase ^= 1;
          return true;
        };
        // S of own block k into the next buffer, once the product that read P there is done
        auto score = [&](int k) {
          const int i = own.off + k * own.step;
          while (at < i)
            if (!skip()) return false;
          if (!mbar_wait_warp(&full[ks], kphase, ab) || !mbar_wait_warp(&odone[2 * t + s_buf], s_phase ^ 1, ab)) return false;
          const uint32_t b = k_lo + ks * (L::kPair >> 4), d = tS + s_buf * 64;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < HD / 16; ++c)
              tc_mma_f16_lo(d, q_lo + (((c / 4) * L::kQBlock + (c % 4) * 32) >> 4), b + (((c / 4) * L::kBlock + (c % 4) * 32) >> 4),
                            kHi, id_s, c > 0);
            tc_commit(&sfull[2 * t + s_buf]);
            if (k + 1 == own.n) tc_commit(qempty);
          }
          __syncwarp();
          s_phase ^= s_buf;
          s_buf ^= 1;
          ++at;
          if (++ks == NS) ks = 0, kphase ^= 1;
          return true;
        };
        if (own.n > 0) {
          if (!(ok = score(0))) break;
        } else {
          if (elect_one()) mbar_arrive(qempty);
          __syncwarp();
        }
#pragma unroll 1
        for (int k = 0; k < own.n; ++k) {
          if (k + 1 < own.n && !(ok = score(k + 1))) break;
          if (!(ok = mbar_wait_warp(&pready[2 * t + p_buf], p_phase, ab))) break;
          tc_fence_after();
          const uint32_t b = v_lo + vs * (L::kPair >> 4), p = tS + p_buf * 64;
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < kKeys / 16; ++c) tc_mma_f16_ts(tO, p + c * 8, b + c * (2048 >> 4), kHi, id_o, k > 0 || c > 0);
            tc_commit(&odone[2 * t + p_buf]);
            tc_commit(&empty[vs]);
          }
          __syncwarp();
          p_phase ^= p_buf;
          p_buf ^= 1;
          vs += own.step;
          if (vs >= NS) vs -= NS;
        }
        while (ok && at < n) ok = skip();
      }
      if (!ok) *ab = 1;
      if (elect_one()) tc_commit(done);  // on every path: arrives once no MMA of this warp is in flight
      __syncwarp();
    }
  } else if (warp >= 12) {
    if constexpr (LOAD) {
      // ---- four warps that load: consecutive lanes take consecutive 16-byte pieces of a row
      constexpr int EB = elem_bytes(CDT), PPR = HD * EB / 16, RSTEP = 128 / PPR, NR = kKeys / RSTEP;
      constexpr int kAhead = Q8 ? L::kRaw - 1 : 2;
      const int lt = threadIdx.x - 384, piece = lt % PPR, row0 = lt / PPR;
      uint8_t* const raw = smem + L::kRawAt;
      int g = 0, landed = 0;     // blocks asked for, and those handed over
      uint32_t edges = 0, gaps = 0;  // of the blocks under way, the last one lowest: edge blocks; this thread's row has no place
      bool ok = true;
      auto wait_slot = [&](int n) { return n < NS || mbar_wait_warp(&empty[n % NS], (n / NS - 1) & 1, ab); };
      // The oldest block under way: its copies have ended for this thread.
      auto hand_over = [&]() {
        const int s = landed % NS, age = g - 1 - landed;
        if constexpr (Q8) {
          if (!wait_slot(landed)) return false;
          const uint8_t* from = raw + (landed % L::kRaw) * L::kRawBytes;
          const bool edge = (edges >> age) & 1;
          bool taken = false;
#pragma unroll
          for (int n = 0; n < 2 * NR; ++n) {
            uint4 w = *reinterpret_cast<const uint4*>(from + (n * 128 + lt) * 16);
            uint32_t* u = reinterpret_cast<uint32_t*>(&w);
            if (edge && n >= NR) {
              uint32_t nan = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) nan |= (u[e] & 0x7F7F7F7Fu) + 0x01010101u;
              if (nan & 0x80808080u) {
                taken = true;
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                  for (int k = 0; k < 32; k += 8)
                    if (((u[e] >> k) & 0x7Fu) == 0x7Fu) u[e] &= ~(0xFFu << k);
              }
            }
            uint32_t f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) f[2 * e] = e4m3x2_to_f16x2(u[e]), f[2 * e + 1] = e4m3x2_to_f16x2(u[e] >> 16);
            const int row = row0 + (n % NR) * RSTEP;
            uint8_t* to = ring + s * L::kPair + (n >= NR ? L::kTile : 0) + row * 128;
            // (lanes of the second 64 elements store their odd piece first: no two of a row's lanes meet in a bank)
            const int odd = HD == 128 ? piece >> 2 : 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int q = 2 * piece + (k ^ odd);
              const uint4 v = (k ^ odd) ? make_uint4(f[4], f[5], f[6], f[7]) : make_uint4(f[0], f[1], f[2], f[3]);
              *reinterpret_cast<uint4*>(to + (q >> 3) * L::kBlock + (((q & 7) ^ (row & 7)) << 4)) = v;
            }
          }
          float sc = *reinterpret_cast<const float*>(from + 2 * kKeys * HD + lt * 4);
          SlotScales& z = s_scale[s];
          if (lt < kKeys) {
            z.k[lt] = sc;
          } else {
            if (edge && !isfinite(sc)) sc = 0.0f, taken = true;
            const float lv = log2_scale_of(sc);
            z.v[lt - kKeys] = sc;
            z.lv[lt - kKeys] = lv;
            float top = lv;
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            if (lane == 0) z.top[warp - 14] = top;
          }
          if (taken) *bad = 1;
        }
        if (warp < 14) {  // positions of the block without a place
          const uint32_t m = __ballot_sync(0xFFFFFFFFu, (gaps >> age) & 1);
          if (lane == 0) {
            reinterpret_cast<uint32_t*>(&hole[s])[warp - 12] = m;
            if (m) *holes = 1;
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        ++landed;
        return true;
      };
      auto flush = [&]() {
        cp_async_wait<0>();
        while (landed < g)
          if (!hand_over()) return false;
        return true;
      };
      for (int it = 0; ok; ++it) {
        const int is = it % kItems;
        // (a piece of work that is not known yet may wait for the blocks under way)
        if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(&ifull[is], (it / kItems) & 1)))
          if (!(ok = flush() && mbar_wait_warp(&ifull[is], (it / kItems) & 1, ab))) break;
        const Item w = items[is];
        __syncwarp();
        if (lane == 0) mbar_arrive(&iempty[is]);
        if (w.stop) break;
        const int first = w.first(), last = w.last(span);
        const ChunkSpan sp = chunk_span(first, last, a.window, a.sinks);
        const int32_t* trow = a.c.table + (int64_t)w.b * a.c.table_width;
        const int in_page = (1 << a.c.log2_page) - 1;
        auto page_of = [&](int pos) {  // -2 where it is not seen by any row, -1 where it has no place
          if (pos > last || (pos < sp.low && pos >= a.sinks)) return -2;
          return paged_page(trow, a.c.table_width, a.c.n_pages, a.c.log2_page, pos);
        };
        int next[NR], next_sc = -2;
        auto look_up = [&](int i) {
          const int kb = chunk_block(sp, i) * kKeys;
#pragma unroll
          for (int n = 0; n < NR; ++n) next[n] = page_of(kb + row0 + n * RSTEP);
          next_sc = page_of(kb + (lt & (kKeys - 1)));
        };
        if (w.i0 < w.i1) look_up(w.i0);
        for (int i = w.i0; i < w.i1; ++i) {
          const int kb = chunk_block(sp, i) * kKeys;
          int page[NR];
#pragma unroll
          for (int n = 0; n < NR; ++n) page[n] = next[n];
          const int page_sc = next_sc;
          if (i + 1 < w.i1) look_up(i + 1);
          if constexpr (!Q8) {
            if (!(ok = wait_slot(g))) break;
          }
          edges = (edges << 1) | (edge_block(kb, first, last, a.window, a.sinks) ? 1u : 0u);
          gaps = (gaps << 1) | (page_sc == -1 ? 1u : 0u);
          if (page_sc == -1) report(a.status, ADP_ERR_INVALID_ARG);
#pragma unroll
          for (int n = 0; n < 2 * NR; ++n) {
            const int row = row0 + (n % NR) * RSTEP, pg = page[n % NR];
            const int64_t cell = (int64_t)max(pg, 0) * a.c.page_bytes +
                                 (int64_t)((w.h << a.c.log2_page) + ((kb + row) & in_page)) * (HD * EB) + piece * 16;
            uint32_t to;
            if constexpr (Q8) {
              to = smem_u32(raw + (g % (Q8 ? L::kRaw : 1)) * L::kRawBytes) + (n * 128 + lt) * 16;
            } else {
              to = smem_u32(ring + (g % NS) * L::kPair) + (n >= NR ? L::kTile : 0) + (piece >> 3) * L::kBlock + row * 128 +
                   (((piece & 7) ^ (row & 7)) << 4);
            }
            cp_async16(to, (n >= NR ? a.c.v : a.c.k) + cell, pg >= 0);
          }
          if constexpr (Q8) {
            const float* from = lt < kKeys ? a.c.k_scale : a.c.v_scale;
            const int64_t cell = (int64_t)max(page_sc, 0) * a.c.scale_stride + (w.h << a.c.log2_page) + ((kb + (lt & (kKeys - 1))) & in_page);
            cp_async4(smem_u32(raw + (g % (Q8 ? L::kRaw : 1)) * L::kRawBytes) + 2 * kKeys * HD + lt * 4, from + cell, page_sc >= 0);
          }
          cp_async_commit();
          ++g;
          if (g - landed > kAhead) {
            cp_async_wait<kAhead>();
            if (!(ok = hand_over())) break;
          }
        }
      }
      if (ok) ok = flush();
      if (!ok) *ab = 1;
      cp_async_wait<0>();
    }
  } else {
    // ---- softmax: warps 0-3 tile A, 4-7 tile B; thread = row = TMEM lane
    const int t = warp >> 2, r = threadIdx.x & 127;
    const int row_tok = r / a.group, row_head = r % a.group;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + t * 128, tO = tmem + lanes + 256 + t * 128;
    bool ok = true;
    uint32_t ns = 0, nh = 0, nq = 0;  // own blocks, items in halves, items with queries so far
    uint32_t g = 0;                   // ring blocks of the items before
    auto wait_all = [&](uint64_t* b, uint32_t parity) { return mbar_wait_warp(b, parity, ab); };
    for (int it = 0; ok; ++it) {
      const int is = it % kItems;
      if (!(ok = wait_all(&ifull[is], (it / kItems) & 1))) break;
      const Item w = items[is];
      if (w.stop) break;
      const int first = w.first(), last = w.last(span), n = w.i1 - w.i0;
      const ChunkSpan sp = chunk_span(first, last, a.window, a.sinks);
      const Own own = own_blocks(w, sp, t, a.tok);
      const bool half = w.half(a.tok);
      const int tok = w.t0 + (half ? 0 : t * a.tok) + row_tok;
      const bool live = r < a.tok * a.group && tok < w.lq;
      const bool warp_live = __any_sync(0xFFFFFFFFu, live);
      const int pos = w.len - w.lq + tok;  // this row's position: it sees keys up to it
      const int from = max(max(pos, 0) - a.window + 1, 0);  // from its window's first on, and the first ones
      const int warp_first = __reduce_min_sync(0xFFFFFFFFu, live ? pos : 0x7FFFFFFF);
      const int warp_last = __reduce_max_sync(0xFFFFFFFFu, live ? pos : -1);
      float scale = a.scale_log2;
      if constexpr (QCONV) {
        // bf16 queries meet fp16 codes: the row is brought to a largest magnitude in [1, 2) by a power of two, so that its
        // 8-bit significands fit fp16 (an element below 2^-17 loses bits: at most 2^-25, half fp16's least step)
        if (n > 0) {
          if (!(ok = wait_all(qfull, nq & 1))) break;
          if (t == 0 || !half) {
            uint8_t* q = Qs + t * L::kQTile + r * 128;
            auto at = [&](int c) { return reinterpret_cast<uint4*>(q + (c / 8) * L::kQBlock + (((c & 7) ^ (r & 7)) << 4)); };
            float top = 0.0f;
#pragma unroll 4
            for (int c = 0; c < HD / 8; ++c) {
              const uint4 v = *at(c);
              const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xFFFF0000u))));
            }
            const uint32_t e2 = min(max(__float_as_uint(top) >> 23, 1u), 253u);
            const float inv = __uint_as_float((254u - e2) << 23);
            if (r < a.tok * a.group) {
#pragma unroll 4
              for (int c = 0; c < HD / 8; ++c) {
                const uint4 v = *at(c);
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                uint32_t f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  f[e] = pack2(__uint_as_float(u[e] << 16) * inv, __uint_as_float(u[e] & 0xFFFF0000u) * inv, DT_F16);
                *at(c) = make_uint4(f[0], f[1], f[2], f[3]);
              }
            }
            s_qf[t * kRows + r] = __uint_as_float(e2 << 23);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(qready);
          if (!(ok = wait_all(qready, nq & 1))) break;
          // (kept finite, as the scale itself)
          scale = fminf(fmaxf(scale * s_qf[half ? r : t * kRows + r], kScaleMin), 3.40282347e38f);
          ++nq;
        }
      }
      // the running maximum (and ms, what is subtracted from scores) and sum, and the score above which the maximum is
      // replaced (never by what stands in rows that are not the sequence's: it must not decide how the others are rounded)
      float m = -INFINITY, ms = 0.0f, l = 0.0f, limit = live ? -INFINITY : INFINITY;
      // e4m3: what weighs V's codes are the products weight x value scale, which have a running maximum of their own, mo
      // (base-2 exponents: score + log2 of the scale); O is relative to it, and vc = 2^(m - mo) brings them there
      float mo = -INFINITY, vc = 1.0f;
      for (int k = 0; k < own.n; ++k, ++ns) {
        const uint32_t buf = ns & 1;
        const int i = own.off + k * own.step;
        if (!(ok = wait_all(&sfull[2 * t + buf], (ns >> 1) & 1))) break;
        tc_fence_after();
        __syncwarp();
        const int slot = (g + i) % NS, kb = chunk_block(sp, w.i0 + i) * kKeys;
        // ---- an edge block's values in 16 bits, looked through by the tiles that weigh them (they take out the same)
        if (!Q8 && edge_block(kb, first, last, a.window, a.sinks)) {
          uint8_t* vt = ring + slot * L::kPair + L::kTile;
          const int key = r >> 1;  // two threads to a key
          auto piece = [&](int c) {
            return reinterpret_cast<uint4*>(vt + (c / 8) * L::kBlock + key * 128 + (((c & 7) ^ (key & 7)) * 16));
          };
          constexpr uint32_t kExp = BF ? 0x7F80u : 0x7C00u, kExp2 = kExp * 0x10001u, kOne2 = (0x8000u - kExp) * 0x10001u;
          if (kb + key >= w.len) {
#pragma unroll
            for (int c = 0; c < HD / 16; ++c) *piece(2 * c + (r & 1)) = make_uint4(0, 0, 0, 0);
          } else {
            // an exponent of all ones carries into its half's sign bit
            uint32_t over = 0;
#pragma unroll
            for (int c = 0; c < HD / 16; ++c) {
              const uint4 v = *piece(2 * c + (r & 1));
              over |= ((v.x & kExp2) + kOne2) | ((v.y & kExp2) + kOne2) | ((v.z & kExp2) + kOne2) | ((v.w & kExp2) + kOne2);
            }
            if (over & 0x80008000u) {
              *bad = 1;
#pragma unroll 1
              for (int c = r & 1; c < HD / 8; c += 2) {
                uint4 v = *piece(c);
                uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  u[e] = ((u[e] & kExp) == kExp ? 0u : u[e] & 0xFFFFu) | ((u[e] & (kExp << 16)) == (kExp << 16) ? 0u : u[e] & 0xFFFF0000u);
                *piece(c) = v;
              }
            }
          }
          fence_async_smem();
          __syncwarp();
        }
        if (warp_live) {
          float x[kKeys];
          tmem_ld64(tS + buf * 64, x);
          const SlotScales& z = s_scale[Q8 ? slot : 0];
          if constexpr (Q8) {
#pragma unroll
            for (int c = 0; c < kKeys; c += 4) {
              const float4 f = *reinterpret_cast<const float4*>(&z.k[c]);
              x[c] *= f.x, x[c + 1] *= f.y, x[c + 2] *= f.z, x[c + 3] *= f.w;
            }
          }
          if (kb + kKeys - 1 > warp_first || (kb <= warp_last - a.window && kb + kKeys - 1 >= a.sinks)) {
            const int left = pos - kb, right = from - kb, few = a.sinks - kb;  // columns c <= left, and c >= right or c < few
#pragma unroll
            for (int c = 0; c < kKeys; ++c) x[c] = c <= left && (c >= right || c < few) ? x[c] : -INFINITY;
          }
          if (*holes) {
            const uint64_t out = *reinterpret_cast<volatile uint64_t*>(&hole[slot]);
#pragma unroll
            for (int c = 0; c < kKeys; ++c) x[c] = (out >> c) & 1 ? -INFINITY : x[c];
          }
          float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int c = 4; c < kKeys - 4; c += 8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) top[e] = max3(top[e], x[c + e], x[c + 4 + e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], x[kKeys - 4 + e]);
          const float mx = max3(fmaxf(top[0], top[1]), top[2], top[3]);
          bool grow = mx > limit;
          if constexpr (Q8) grow |= live && mx > -INFINITY && fmaf(mx, scale, fmaxf(z.top[0], z.top[1])) > mo + kRescale;
          if (__any_sync(0xFFFFFFFFu, grow)) {
            const float mn = live && mx > -INFINITY ? fmaxf(m, mx * scale) : m;
            float f = mn == -INFINITY ? 1.0f : exp2_fast(m - mn);
            m = mn;
            ms = m == -INFINITY ? 0.0f : m - kWeightUp<BF>;
            l *= f;
            if (live && m > -INFINITY) limit = (m + kRescale) / scale;
            if constexpr (Q8) {  // (both maxima at once: mo is m - 126 at least, and vc finite)
              float mw = -INFINITY;
#pragma unroll
              for (int c = 0; c < kKeys; c += 4) {
                const float4 lv = *reinterpret_cast<const float4*>(&z.lv[c]);
                mw = fmaxf(fmaxf(mw, fmaf(x[c], scale, lv.x)), fmaf(x[c + 1], scale, lv.y));
                mw = fmaxf(fmaxf(mw, fmaf(x[c + 2], scale, lv.z)), fmaf(x[c + 3], scale, lv.w));
              }
              mw = live ? fmaxf(mo, mw) : mo;
              f = mw == -INFINITY ? 1.0f : exp2_fast(mo - mw);
              mo = mw;
              vc = mw == -INFINITY ? 1.0f : exp2_fast(m - mw);
            }
            if (k > 0) {
              // own block k - 1's product must be in O
              if (!(ok = wait_all(&odone[2 * t + (buf ^ 1)], ((ns - 1) >> 1) & 1))) break;
              tc_fence_after();
#pragma unroll 1
              for (int c0 = 0; c0 < HD; c0 += 32) {
                float o[32];
                tmem_ld32(tO + c0, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= f;
                tmem_st32(tO + c0, o);
              }
            }
          }
          const float2 sc = make_float2(scale, scale), nm = make_float2(-ms, -ms);
          float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
          for (int c0 = 0; c0 < kKeys; c0 += 32) {
            uint32_t u[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 y = __ffma2_rn(make_float2(x[c0 + e], x[c0 + e + 1]), sc, nm);
              float2 p = make_float2(exp2_fast(y.x), exp2_fast(y.y));  // (0 where x is -infinity: not seen)
              sum[(e >> 1) & 1] = __fadd2_rn(sum[(e >> 1) & 1], p);
              if constexpr (Q8) {  // (cut where the weight is 0 next to it, or as good as: 0 times infinity is none)
                const float2 f = *reinterpret_cast<const float2*>(&z.v[c0 + e]);
                p.x *= min_nan(f.x * vc, kFactorMax);
                p.y *= min_nan(f.y * vc, kFactorMax);
              }
              u[e >> 1] = pack2(p.x, p.y, BF ? DT_BF16 : DT_F16);
            }
            tmem_st16(tS + buf * 64 + c0 / 2, u);
          }
          tmem_st_wait();
          tc_fence_before();
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[2 * t + buf]);
      }
      // ---- behind the last two products (the others' ends were waited for when S took their P's place)
      if (ok && own.n > 1) ok = wait_all(&odone[2 * t + (ns & 1)], ((ns - 2) >> 1) & 1);
      if (ok && own.n > 0) ok = wait_all(&odone[2 * t + (~ns & 1)], ((ns - 1) >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      g += n;
      const float out_of = Q8 && mo > -INFINITY ? 0.5f * (mo - m) : 0.0f;  // O is relative to mo (brought to m in two steps)
      float own_f = exp2_fast(out_of), other_f = 0.0f;
      bool other = false;
      if (half && n > 1) {
        if (t == 1) {
          s_half[r] = m;
          s_half[kRows + r] = l;
          if constexpr (Q8) s_half[2 * kRows + r] = own_f;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(hfull);
          if (!(ok = wait_all(hfree, nh & 1))) break;
          tc_fence_after();
        } else {
          if (!(ok = wait_all(hfull, nh & 1))) break;
          tc_fence_after();
          other = true;
        }
        ++nh;
      }
      if (t == 0 || !half) {
        float fb = 0.0f, fa = 1.0f;
        if (other) {
          const float mb = s_half[r], top = fmaxf(m, mb), base = top == -INFINITY ? 0.0f : top;
          other_f = Q8 ? s_half[2 * kRows + r] : 1.0f;
          fa = exp2_fast(m - base);
          fb = exp2_fast(mb - base);
          l = fmaf(l, fa, s_half[kRows + r] * fb);
          m = top;
        }
        const float inv = w.part >= 0 ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
        uint8_t* po = a.out + (int64_t)(w.q0 + tok) * a.out_stride + (int64_t)(w.h * a.group + row_head) * HD * 2;
        const int64_t prow = w.part >= 0 ? ((int64_t)blockIdx.x * 2 + w.part) * a.rows_cap + t * kRows + r : 0;
        if (w.part >= 0 && live) a.part_ml[prow] = make_float2(m, l);
        if (warp_live) {
#pragma unroll 1
          for (int c0 = 0; c0 < HD; c0 += 32) {
            float o[32];
            if (own.n > 0) {
              tmem_ld32(tO + c0, o);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0.0f;
            }
            if (Q8 || other) {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = o[e] * own_f * own_f * fa;
            }
            if (other) {
              float q[32];
              tmem_ld32(tO + 128 + c0, q);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = fmaf(q[e] * other_f * other_f, fb, o[e]);
            }
            if (live) {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = l == 0.0f ? 0.0f : o[e] * inv;
              if (*bad) {  // what was taken out of edge blocks comes to the rows that see it
                for (int i = w.i0; i < w.i1; ++i) {
                  const int kb = chunk_block(sp, i) * kKeys;
                  if (!edge_block(kb, first, last, a.window, a.sinks)) continue;
                  for (int key = kb; key < kb + kKeys && key <= pos; ++key) {
                    if (key < from && key >= a.sinks) continue;
                    const int page = paged_page(a.c.table + (int64_t)w.b * a.c.table_width, a.c.table_width, a.c.n_pages, a.c.log2_page, key);
                    if (page < 0) continue;
                    const int cell = (w.h << a.c.log2_page) + (key & ((1 << a.c.log2_page) - 1));
                    const uint8_t* pv = a.c.v + (int64_t)page * a.c.page_bytes + ((int64_t)cell * HD + c0) * elem_bytes(CDT);
                    const float f = Q8 ? a.c.v_scale[(int64_t)page * a.c.scale_stride + cell] : 1.0f;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                      float v = load_elem(pv, e, CDT);
                      if (Q8) v *= f;
                      o[e] += isfinite(v) ? 0.0f : v;
                    }
                  }
                }
              }
              if (w.part >= 0) {
                float4* to = reinterpret_cast<float4*>(a.part_o + prow * HD + c0);
#pragma unroll
                for (int e = 0; e < 32; e += 4) to[e / 4] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
              } else {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                  uint32_t u[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k) u[k] = pack2(o[e + 2 * k], o[e + 2 * k + 1], QDT);
                  *reinterpret_cast<uint4*>(po + (c0 + e) * 2) = make_uint4(u[0], u[1], u[2], u[3]);
                }
              }
            }
            __syncwarp();
          }
        }
        if (other) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(hfree);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&iempty[is]);
    }
    if (!ok) {
      *ab = 1;
      if (r == 0) report(a.status, ADP_ERR_PIPELINE_TIMEOUT);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // no MMA may be in flight (nor TMEM in use) when the accumulators are freed
  if (warp == 9) mbar_wait(done, 0, &never, a.wait_ns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Joins the pieces that several CTAs share: block (c, y) takes the piece that starts in CTA c and goes on behind it, and 8 of
// its rows, a warp each.
template <int HD, int QDT>
__global__ void __launch_bounds__(256) paged_chunk_join_kernel(const ChunkArgs a) {
  constexpr int W = HD / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const ChunkMeta meta = a.meta[blockIdx.x];
  const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int tile = r / kRows, rr = r % kRows, tok = tile * a.tok + rr / a.group;
  if (!meta.starts || rr >= a.tok * a.group || tok >= meta.tokens) return;
  const int ctas = (int)gridDim.x + 1;
  float m = -INFINITY, l = 0.0f, o[W];
#pragma unroll
  for (int e = 0; e < W; ++e) o[e] = 0.0f;
  auto add = [&](int64_t row) {
    const float2 ml = a.part_ml[row];
    const float mn = fmaxf(m, ml.x), base = mn == -INFINITY ? 0.0f : mn;
    const float f = exp2_fast(m - base), g = exp2_fast(ml.x - base);
    m = mn;
    l = fmaf(l, f, g * ml.y);
#pragma unroll
    for (int e = 0; e < W; ++e) o[e] = fmaf(o[e], f, g * a.part_o[row * HD + e * 32 + lane]);
  };
  add(((int64_t)blockIdx.x * 2 + 1) * a.rows_cap + r);
  for (int c0 = (int)blockIdx.x + 1; c0 < ctas; c0 += 32) {
    const int first = c0 + lane < ctas ? a.meta[c0 + lane].first : 0;
    const uint32_t ends = __ballot_sync(0xFFFFFFFFu, first == 2);
    uint32_t has = __ballot_sync(0xFFFFFFFFu, first != 0);
    if (ends) has &= (ends ^ (ends - 1));  // up to the first end
    for (; has; has &= has - 1) add((int64_t)(c0 + __ffs(has) - 1) * 2 * a.rows_cap + r);
    if (ends) break;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint8_t* po = a.out + (int64_t)(meta.row0 + tok) * a.out_stride + (int64_t)(meta.head * a.group + rr % a.group) * HD * 2;
#pragma unroll
  for (int e = 0; e < W; ++e)
    reinterpret_cast<uint16_t*>(po)[e * 32 + lane] = round_kv(l == 0.0f ? 0.0f : o[e] * inv, QDT);
}

// ---------------------------------------------------------------- host side

// Pages of a pool as boxes of 64 elements x the rows of a page (at most 64).
bool encode_pages(CUtensorMap* map, const void* base, bool bf16, const adp_paged_kv* kv) {
  const cuuint64_t dims[4] = {(cuuint64_t)kv->head_dim, (cuuint64_t)kv->page_size, (cuuint64_t)kv->n_kv_heads, (cuuint64_t)kv->n_pages};
  const cuuint64_t row = (cuuint64_t)kv->head_dim * 2;
  const cuuint64_t strides[3] = {row, row * kv->page_size, (cuuint64_t)kv->page_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)(kv->page_size < kKeys ? kv->page_size : kKeys), 1, 1}, one[4] = {1, 1, 1, 1};
  return encode_fn()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(base),
                     dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMinCopyPage = 8;  // positions of a page that a tensor copy takes: whole swizzle atoms

// How a call falls on the GPU: CTAs, rows of a partial result (0: no piece of work can be cut), bytes of the workspace.
struct ChunkPlan {
  int ctas, rows_cap;
  size_t bytes;
};

ChunkPlan chunk_plan(const adp_paged_kv* kv, int group, int n_rows, int sms, int32_t window, int32_t sinks) {
  const int tok = kRows / group, span = 2 * tok;
  // at most: every sequence may end inside a pair, fill its table, and its window may start inside a block
  const int64_t items = ((int64_t)n_rows / span + (kv->n_seqs < n_rows ? kv->n_seqs : n_rows)) * kv->n_kv_heads;
  const int64_t all = ((int64_t)kv->table_width * kv->page_size + kKeys - 1) / kKeys;
  const int64_t seen = ((int64_t)window + span + kKeys - 2) / kKeys + 1 + ((int64_t)sinks + kKeys - 1) / kKeys;
  const int64_t blocks = seen < all ? seen : all;
  ChunkPlan p{};
  p.ctas = chunk_parts(items * (blocks + kChunkOver), items, sms);
  if (blocks >= 2 * kChunkMinPart && p.ctas > 1) {
    p.rows_cap = n_rows <= tok ? kRows : 2 * kRows;
    p.bytes = (size_t)p.ctas * (2 * p.rows_cap * ((size_t)kv->head_dim * sizeof(float) + sizeof(float2)) + sizeof(ChunkMeta));
  }
  return p;
}

template <int HD, int CDT, int QDT, bool LOAD>
struct ChunkKey {};

template <int HD, int CDT, int QDT, bool LOAD>
cudaError_t chunk_launch(const CUtensorMap (&m)[3], const ChunkArgs& a, const ChunkPlan& p, cudaStream_t st) {
  auto* kernel = paged_chunk_kernel<HD, CDT, QDT, LOAD>;
  constexpr size_t smem = ChunkSmem<HD, CDT>::kBytes;
  cudaError_t e = allow_smem<ChunkKey<HD, CDT, QDT, LOAD>>((const void*)kernel, smem);
  if (e != cudaSuccess) return e;
  kernel<<<p.ctas, LOAD ? 512 : 384, smem, st>>>(m[0], m[1], m[2], a);
  if ((e = cudaGetLastError()) != cudaSuccess || !p.rows_cap) return e;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.ctas - 1, p.rows_cap / 8);  // no piece goes on behind the last CTA
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_chunk_join_kernel<HD, QDT>, a);
}

int chunk_check(const adp_paged_kv* kv, int32_t n_heads, int32_t n_rows, int32_t window, int32_t sinks, PagedView* c) {
  const int rc = paged_view(kv, c);
  if (rc) return rc;
  if (n_heads < 1 || n_heads % kv->n_kv_heads || n_rows < 0 || window < 0 || sinks < 0) return ADP_ERR_INVALID_ARG;
  if (n_heads / kv->n_kv_heads > kRows || n_heads > 65536 || kv->n_seqs > kPagedMaxSeqs) return ADP_ERR_UNSUPPORTED_CONFIG;
  return ADP_OK;
}

}  // namespace
}  // namespace adp

using namespace adp;

extern "C" int adp_paged_chunk_attention_workspace(const adp_paged_kv* kv, int32_t n_heads, int32_t n_rows, int32_t window,
                                                   int32_t sinks, uint64_t* bytes) {
  PagedView c;
  int rc = bytes ? chunk_check(kv, n_heads, n_rows, window, sinks, &c) : ADP_ERR_INVALID_ARG;
  int sms = 0;
  if (rc || (rc = sm_count(&sms))) return rc;
  *bytes = chunk_plan(kv, n_heads / kv->n_kv_heads, n_rows, sms, window ? window : kNoWindow, sinks).bytes;
  return ADP_OK;
}

extern "C" int adp_paged_chunk_attention(const adp_paged_kv* kv, const void* q, int32_t q_dtype, int32_t n_heads,
                                         int64_t q_stride, const int32_t* cu_rows, int32_t n_rows, float scale, int32_t window,
                                         int32_t sinks, void* out, int64_t out_stride, void* workspace,
                                         uint64_t workspace_bytes, int32_t* dev_status, void* cuda_stream) {
  ChunkArgs a{};
  int rc = chunk_check(kv, n_heads, n_rows, window, sinks, &a.c);
  if (rc) return rc;
  if (q_dtype != ADP_F16 && q_dtype != ADP_BF16) return ADP_ERR_UNSUPPORTED_CONFIG;
  if (kv->dtype != ADP_E4M3 && kv->dtype != q_dtype) return ADP_ERR_UNSUPPORTED_CONFIG;
  if (!isfinite(scale) || !cu_rows || ((uintptr_t)cu_rows & 3) || ((uintptr_t)dev_status & 3)) return ADP_ERR_INVALID_ARG;
  if (kv->n_seqs == 0 || n_rows == 0) return ADP_OK;
  const int64_t width = (int64_t)n_heads * kv->head_dim;
  if (!q || !out || !aligned16(q) || !aligned16(out) || q_stride < width || out_stride < width || q_stride % 8 || out_stride % 8)
    return ADP_ERR_INVALID_ARG;
  int sms = 0;
  if ((rc = sm_count(&sms))) return rc;
  const int group = n_heads / kv->n_kv_heads;
  a.window = window ? window : kNoWindow;
  a.sinks = sinks;
  const ChunkPlan plan = chunk_plan(kv, group, n_rows, sms, a.window, sinks);
  if (plan.bytes && (!workspace || !aligned16(workspace) || workspace_bytes < plan.bytes)) return ADP_ERR_INVALID_ARG;
  if (!encode_fn()) return cuda_status(cudaErrorNotSupported, "cuTensorMapEncodeTiled");
  const bool bf16 = q_dtype == ADP_BF16, load = kv->dtype == ADP_E4M3 || kv->page_size < kMinCopyPage;
  a.cu = cu_rows;
  a.out = static_cast<uint8_t*>(out);
  a.out_stride = out_stride * 2;
  a.n_rows = n_rows;
  a.group = group;
  a.tok = kRows / group;
  // (a scale of 0 becomes the least normal number: the scores' differences vanish all the same, and what is not seen stays at
  // -infinity)
  a.scale_log2 = fmaxf(log2_scale(fabsf(scale)), kScaleMin);
  a.neg = scale < 0.0f ? kTcIdescANeg : 0;
  a.rows_cap = plan.rows_cap;
  if (plan.bytes) {
    const size_t rows = (size_t)plan.ctas * 2 * plan.rows_cap;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + rows * kv->head_dim);
    a.meta = reinterpret_cast<ChunkMeta*>(a.part_ml + rows);
  }
  a.status = dev_status;
  const int64_t keys = (int64_t)kv->table_width * kv->page_size;
  a.wait_ns = packed_wait_ns((int32_t)keys, kv->n_seqs);
  CUtensorMap m[3] = {};
  if (!encode(&m[0], q, bf16, kv->head_dim, n_heads, n_rows, q_stride, group, a.tok)) return ADP_ERR_INVALID_ARG;
  if (!load && (!encode_pages(&m[1], kv->k, bf16, kv) || !encode_pages(&m[2], kv->v, bf16, kv))) return ADP_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaErrorInvalidValue;
  using F = std::integral_constant<int, DT_F16>;
  using B = std::integral_constant<int, DT_BF16>;
  using E = std::integral_constant<int, DT_E4M3>;
  auto go = [&](auto hd, auto cdt, auto qdt, auto l) {
    e = chunk_launch<decltype(hd)::value, decltype(cdt)::value, decltype(qdt)::value, decltype(l)::value>(m, a, plan, st);
  };
  auto by_type = [&](auto hd) {
    if (kv->dtype == ADP_E4M3) {
      if (bf16) go(hd, E(), B(), std::true_type());
      else go(hd, E(), F(), std::true_type());
    } else if (bf16) {
      if (load) go(hd, B(), B(), std::true_type());
      else go(hd, B(), B(), std::false_type());
    } else {
      if (load) go(hd, F(), F(), std::true_type());
      else go(hd, F(), F(), std::false_type());
    }
  };
  if (kv->head_dim == 128) by_type(std::integral_constant<int, 128>());
  else by_type(std::integral_constant<int, 64>());
  return cuda_status(e, "adp_paged_chunk_attention");
}
