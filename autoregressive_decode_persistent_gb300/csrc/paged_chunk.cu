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
constexpr int kItems = 2;               // the piece of work and the next one

// What a range of work says of its first part of a piece (a word in global memory): nothing yet, the part is written and goes on in
// the next range, it is written and ends there, or the range has none.
enum PartState : int32_t { kPartOpen = 0, kPartGoesOn = 1, kPartEnds = 2, kPartNone = 3 };

struct ChunkArgs {
  PagedView c;
  const int32_t* cu;
  uint8_t* out;
  int64_t out_stride;            // bytes
  int32_t n_rows, group, tok;    // query heads per KV head; tokens of a tile
  int32_t window, sinks;
  float scale_log2;              // of |scale|, and above 0
  int32_t even_scales;           // e4m3: four positions' scales are 16 aligned bytes wherever their pages lie
  uint32_t neg;                  // scale < 0: the instruction descriptor's bit that negates A
  int32_t rows_cap;              // rows of a partial result (128 or 256)
  float* part_o;                 // [ctas][rows_cap / 32][head_dim / 4][32 rows][4]
  float2* part_ml;               // [ctas][rows_cap]
  int32_t* part_state;           // [ctas], PartState
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
  int32_t part;  // -1: all of its blocks; 0: a part that goes on from the range before; 1: the first part of several
  int32_t stop;  // no work is left
  __device__ __forceinline__ int first() const { return len - lq + t0; }
  __device__ __forceinline__ int last(int span) const { return len - lq + min(t0 + span, lq) - 1; }
  // its rows fit one tile: the tiles take turns at the blocks
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
// The bits below n of 64.
__device__ __forceinline__ uint64_t below(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }

// Whether some row of the item does not see all positions of the block at position kb.
__device__ __forceinline__ bool edge_block(int kb, int first, int last, int window, int sinks) {
  return kb + kKeys - 1 > first || (kb <= last - window && kb + kKeys - 1 >= sinks);
}

// The table's entry for a position (any position at or behind 0), and the page that it names: -2 where none of the n positions
// from pos on, all in one page, is seen by a row, -1 where it names none.
__device__ __forceinline__ int table_entry(const ChunkArgs& a, const int32_t* row, int pos) {
  return __ldg(row + min(pos >> a.c.log2_page, a.c.table_width - 1));
}
__device__ __forceinline__ int page_of(const ChunkArgs& a, int entry, int pos, int n, int low, int last) {
  if (pos > last || (pos + n <= low && pos >= a.sinks)) return -2;
  return entry >= 0 && entry < a.c.n_pages ? entry : -1;
}

// The line of all work: KV heads, in them sequences, in them pairs of tiles of tokens, in them blocks.
struct Place {
  int32_t h, b, t, j;  // KV head, sequence, pair, block
  __device__ __forceinline__ bool before(const Place& o) const {
    return h != o.h ? h < o.h : b != o.b ? b < o.b : t != o.t ? t < o.t : j < o.j;
  }
};

__device__ __forceinline__ int pair_blocks(const ChunkArgs& a, const Rows& r, int t) {
  const int span = 2 * a.tok, first = r.len - r.lq + t * span, last = r.len - r.lq + min((t + 1) * span, r.lq) - 1;
  return chunk_span(first, last, a.window, a.sinks).n;
}
__device__ __forceinline__ int pair_units(const ChunkArgs& a, const Rows& r, int t) {
  return pair_blocks(a, r, t) + chunk_over(r.lq - t * 2 * a.tok, a.tok);
}
__device__ __forceinline__ Rows shfl_rows(const Rows& r, int l) {
  return Rows{__shfl_sync(0xFFFFFFFFu, r.q0, l), __shfl_sync(0xFFFFFFFFu, r.lq, l), __shfl_sync(0xFFFFFFFFu, r.len, l)};
}
// Units of a sequence for one KV head, one lane per sequence; long ones are added up by the whole warp.
__device__ __forceinline__ int64_t sequence_units(const ChunkArgs& a, const Rows& r, int lane) {
  constexpr int kAlone = 2;
  const int span = 2 * a.tok, pairs = (r.lq + span - 1) / span;
  int64_t sum = 0;
  if (pairs <= kAlone)
    for (int t = 0; t < pairs; ++t) sum += pair_units(a, r, t);
  for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, pairs > kAlone); todo; todo &= todo - 1) {
    const int l = __ffs(todo) - 1, n = __shfl_sync(0xFFFFFFFFu, pairs, l);
    const Rows o = shfl_rows(r, l);
    int64_t s = 0;
    for (int t = lane; t < n; t += 32) s += pair_units(a, o, t);
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
// Units and pairs of 32 sequences, for one KV head.
struct Units {
  int64_t units;
  int32_t pairs;
};

// The warp that finds the work: its lanes hold 32 sequences at a time.
struct Finder {
  const ChunkArgs& a;
  const int lane, span;
  int chunk;       // the sequences held: from 32 x chunk on
  Rows mine;
  int64_t units, upto;  // of this lane's sequence, and with those before it
  __device__ __forceinline__ Finder(const ChunkArgs& args, int l) : a(args), lane(l), span(2 * args.tok), chunk(-1), mine{0, 0, 0}, units(0), upto(0) {}
  __device__ __forceinline__ void hold(int ch, int32_t* status) {
    if (ch == chunk) return;
    chunk = ch;
    mine = Rows{0, 0, 0};
    if (ch * 32 + lane < a.c.n_seqs) mine = rows_of(a, ch * 32 + lane, status);
  }
  __device__ __forceinline__ void add_up() {
    units = sequence_units(a, mine, lane);
    upto = scan_inclusive(units, lane);
  }
  __device__ __forceinline__ int pairs() const { return (mine.lq + span - 1) / span; }
  // Where a cut at unit x of a head's line goes, within the sequences held (and added up).
  __device__ __forceinline__ Place place(int h, int64_t x) const {
    const int l = min(__popc(__ballot_sync(0xFFFFFFFFu, upto <= x)), 31);
    x -= __shfl_sync(0xFFFFFFFFu, upto - units, l);
    const Rows o = shfl_rows(mine, l);
    const int n = (o.lq + span - 1) / span;
    for (int t0 = 0; t0 < n; t0 += 32) {
      const int blocks = t0 + lane < n ? pair_blocks(a, o, t0 + lane) : 0;
      const int64_t own = t0 + lane < n ? pair_units(a, o, t0 + lane) : 0, sum = scan_inclusive(own, lane);
      const int p = __popc(__ballot_sync(0xFFFFFFFFu, sum <= x));
      if (p == 32) {
        x -= __shfl_sync(0xFFFFFFFFu, sum, 31);
        continue;
      }
      x -= __shfl_sync(0xFFFFFFFFu, sum - own, p);
      return Place{h, chunk * 32 + l, t0 + p, chunk_cut(__shfl_sync(0xFFFFFFFFu, blocks, p), x - chunk_over(o.lq - (t0 + p) * span, a.tok))};
    }
    return Place{h, chunk * 32 + l, n, 0};  // (the offsets changed while this call ran)
  }
};

// Per ring slot of e4m3 blocks: the scales, log2 of the value scales and its largest over each half of the block.
struct SlotScales {
  float k[kKeys], v[kKeys], lv[kKeys], top[4];
};

__device__ __forceinline__ void say_part(const ChunkArgs& a, int range, int32_t state) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(a.part_state + range), "r"(state) : "memory");
}
__device__ __forceinline__ int32_t part_said(const ChunkArgs& a, int range) {
  int32_t v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(a.part_state + range) : "memory");
  return v;
}

template <int HD, int CDT>
struct ChunkSmem {
  static constexpr bool kConv = CDT == DT_E4M3;
  static constexpr int kSlots = HD == 64 ? 8 : kConv ? 3 : 4;  // of a block of K and one of V
  static constexpr int kRaw = kConv ? (HD == 128 ? 5 : 8) : 0;   // blocks of codes of K or of V under way
  static constexpr uint32_t kQBlock = 128 * 128;            // 128 rows x 64 elements, swizzled
  static constexpr uint32_t kQTile = (HD / 64) * kQBlock;
  static constexpr uint32_t kBlock = kKeys * 128;           // the same of K or V
  static constexpr uint32_t kTile = (HD / 64) * kBlock;
  static constexpr uint32_t kPair = 2 * kTile;
  static constexpr int kOutBytes = kConv ? 64 : 128;        // of a row of results on their way out
  static constexpr int kOutCols = kOutBytes / 8;            // columns of results that tiles and warps add up at a time, in two buffers
  static constexpr uint32_t kRawBytes = kKeys * HD + kKeys * 4;  // codes, and a scale for each row
  static constexpr uint32_t kRawAt = 2 * kQTile + kSlots * kPair;
  static constexpr uint32_t kOut = kRawAt + kRaw * kRawBytes;
  static constexpr uint32_t kScales = kOut + 8 * 32 * kOutBytes;                           // [kSlots], e4m3
  static constexpr uint32_t kQf = kScales + (kConv ? kSlots * sizeof(SlotScales) : 0);     // [256] of the rows of Q, e4m3
  static constexpr uint32_t kHalf = kQf + (kConv ? 2 * kRows * 4 : 0);                     // [2][256]
  static constexpr uint32_t kCtl = kHalf + 4 * kRows * 4;
  static constexpr uint32_t kCtlBytes = kConv ? 768 : 512;
  static constexpr size_t kBytes = kCtl + kCtlBytes;
};

// LOAD: registers of a thread of the softmax warps, of those that find, copy and issue, and of those that load; the four groups of
// 128 threads start with 128 each.
constexpr int kSoftmaxRegs = 160, kIssueRegs = 72, kLoadRegs = 120;
static_assert(2 * kSoftmaxRegs + kIssueRegs + kLoadRegs == 4 * 128, "what is taken has to be given");
template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Four e4m3 codes as fp16 (exact): the low pair and the high pair.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
// Copy of consecutive bytes (a multiple of 16, from and to multiples of 16) into this CTA's shared memory, completing on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ uint4 zero_codes[kKeys * 128 / 16];  // what is read where a block's positions have no place
__device__ __forceinline__ float log2_scale_of(float s) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fabsf(s)));
  return fmaxf(y, -126.0f);  // (2^-126: the least scale there is)
}
// What was taken out of the values (of blocks lo .. hi, by their positions) and is seen by a row: the sum for 4 columns from col on.
template <int HD, int CDT>
__device__ __forceinline__ float4 taken_out(const ChunkArgs& a, const Item& w, int pos, int col, int lo, int hi) {
  const int first = w.first(), last = w.last(2 * a.tok), from = max(max(pos, 0) - a.window + 1, 0);
  const ChunkSpan sp = chunk_span(first, last, a.window, a.sinks);
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = w.i0; i < w.i1; ++i) {
    const int kb = chunk_block(sp, i) * kKeys;
    if (kb < lo || kb > hi || !edge_block(kb, first, last, a.window, a.sinks)) continue;
    for (int key = kb; key < kb + kKeys && key <= pos; ++key) {
      if (key < from && key >= a.sinks) continue;
      const int page = paged_page(a.c.table + (int64_t)w.b * a.c.table_width, a.c.table_width, a.c.n_pages, a.c.log2_page, key);
      if (page < 0) continue;
      const int at = (w.h << a.c.log2_page) + (key & ((1 << a.c.log2_page) - 1));
      const uint8_t* pv = a.c.v + (int64_t)page * a.c.page_bytes + (int64_t)at * HD * elem_bytes(CDT);
      const float f = CDT == DT_E4M3 ? a.c.v_scale[(int64_t)page * a.c.scale_stride + at] : 1.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = load_elem(pv, col + e, CDT);
        if (CDT == DT_E4M3) v *= f;
        sum[e] += isfinite(v) ? 0.0f : v;
      }
    }
  }
  return make_float4(sum[0], sum[1], sum[2], sum[3]);
}

// Every sequence's last rows over its pages.  Per row and block of 64 positions: S = q K^T; with the running maximum m of the
// row's scores (kept while it is within 2^8 of what it would be), P = 2^(scale S - m), l += sum P, O += P V; at the end O / l.  Parts of
// a row's positions have an (m, l, O) of their own and are joined by O = sum_i 2^(m_i - m) O_i, l likewise.
//
// Rows of a tile are tokens x query heads of one KV head (128 rows: K and V are read once for the heads that share them).  An
// item of work is two tiles and the blocks that they see; S and O lie in TMEM, Q and a ring of K and V in shared memory, and a
// thread of the softmax warps has a row.  Where the rows fit one tile, the tiles take turns at the blocks, and maxima, sums and results are
// added up at the end (quarters of a block's positions for each warp of a tile, where the rows fit a warp, were slower: 16 rows
// over 77 positions 12.3 us for 10.3, 32 sequences of up to 8 rows over 16 bits 111 for 105).  The line of all items (KV heads, in them
// sequences, pairs of tiles, blocks) is cut evenly over the SMs, whatever the lengths: the CTA that starts an item joins what
// the next ones have of it.
//
// Measured: long chunks are bound by the MMAs and the softmax warps, which both fill most of a block's time (2,048 rows of 32/8
// heads x 128 over 8,192 bf16 positions: 241 GFLOP in 181 us, 70% of the GEMM rate, the tensor pipe busy 57% of it; some
// 1,280 cycles of a pair's block, 1,024 by the pipe's rate: S's 64 columns read Q again for every block).  Few rows over 16 bits are
// bound by memory (32 sequences of 4 rows, 8,192 positions each: 1.07 GB in 178 us, 89% of the copy rate), over e4m3
// by a block's way from codes to O, on which two tiles and three slots of fp16 blocks keep two blocks at a time, 0.8 us each (the
// same in e4m3: 206 us, 40%; with three quarters of the conversions left out 32 sequences of up to 8 rows took 144 us for 146).
//
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
  // (there is no room to align it by hand, and no need: no other shared memory lies in front)
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    report(a.status, ADP_ERR_CUDA);
    return;
  }
  uint8_t* Qs = smem;
  uint8_t* ring = smem + 2 * L::kQTile;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kCtl);
  uint64_t* full = bar;               // [NS]
  uint64_t* empty = full + NS;        // [NS]
  uint64_t* qfull = empty + NS;
  uint64_t* qready = qfull + 1;       // (QCONV)
  uint64_t* qempty = qready + 1;
  uint64_t* joined = qempty + 1;      // the softmax warps meet
  uint64_t* done = joined + 1;
  uint64_t* sfull = done + 1;         // [2][2]: tile, buffer
  uint64_t* pready = sfull + 4;       // [2][2]
  uint64_t* odone = pready + 4;       // [2][2]
  uint64_t* ifull = odone + 4;        // [kItems]
  uint64_t* iempty = ifull + kItems;  // [kItems]
  uint64_t* vfull = iempty + kItems;       // [NS] e4m3: the block's V (and full: its K)
  uint64_t* rawfull = vfull + (Q8 ? NS : 0);  // [kRaw]
  uint64_t* rawempty = rawfull + L::kRaw;  // [kRaw]
  uint64_t* rawhole = rawempty + L::kRaw;  // [kRaw], as hole
  uint64_t* hole = rawhole + L::kRaw;      // [NS]: positions of the block whose page has no place
  int32_t* ctl = reinterpret_cast<int32_t*>(hole + NS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctl);
  volatile int32_t* ab = ctl + 1;
  volatile int32_t* holes = ctl + 2;  // some block had a position without a page
  int32_t* taken = ctl + 6;           // positions of the first and of the last block that a non-finite value was taken out of
  Item* items = reinterpret_cast<Item*>(ctl + 8);  // [kItems]
  float* s_half = reinterpret_cast<float*>(smem + L::kHalf);  // where tiles and warps share rows: maxima and sums
  float* s_qf = reinterpret_cast<float*>(smem + L::kQf);
  SlotScales* s_scale = reinterpret_cast<SlotScales*>(smem + L::kScales);
  static_assert(((Q8 ? 4 : 3) * NS + 21 + 3 * L::kRaw) * 8 + 32 + kItems * sizeof(Item) <= L::kCtlBytes, "the control words' room");
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], Q8 ? 2 : LOAD ? 4 : 1);
      mbar_init(&empty[s], 2);  // tiles
      if constexpr (Q8) mbar_init(&vfull[s], 2);
      hole[s] = 0;
    }
    mbar_init(qfull, 1);
    mbar_init(qready, 8);
    mbar_init(qempty, 2);
    mbar_init(joined, 8);
    mbar_init(done, 2);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pready[i], 4);  // warps
      mbar_init(&odone[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&ifull[i], 1);
      mbar_init(&iempty[i], 10 + (LOAD ? 4 : 0) + (!LOAD || Q8 ? 1 : 0));  // the issuing and the softmax warps, those that load
    }
    for (int i = 0; i < L::kRaw; ++i) {
      mbar_init(&rawfull[i], 1);
      mbar_init(&rawempty[i], 2);
    }
    *ab = 0;
    *holes = 0;
    taken[0] = 0x7FFFFFFF;
    taken[1] = -1;
    ctl[3] = (int32_t)(a.wait_ns >> 19 < 0x7FFFFFFF ? a.wait_ns >> 19 : 0x7FFFFFFF);  // (2^20 cycles are 2^19 ns and more)
    *reinterpret_cast<uint64_t*>(ctl + 4) = a.wait_ns;
    mbar_fence_init();
  }
  // A range's last piece is joined by the CTA that starts it, which waits for the next range's beginning: that range belongs to a CTA
  // with a lower number, which is launched no later.  (So this GPU does it; the programming model does not promise it, and the wait
  // is bounded: a CTA that gives up reports it, and its rows stay unset.)
  const int range = (int)(gridDim.x - 1 - blockIdx.x);
  // ---- units and pairs of every 32 sequences (one warp's worth: the finding warp adds them up alone)
  const int n_chunks = (a.c.n_seqs + 31) / 32, span = 2 * a.tok;
  Units* chunks = reinterpret_cast<Units*>(smem);  // [n_chunks] (before anything is copied there)
  if (n_chunks > 1) {
    for (int ch = warp; ch < n_chunks; ch += kWarps) {
      Rows r{0, 0, 0};
      if (ch * 32 + lane < a.c.n_seqs) r = rows_of(a, ch * 32 + lane, a.status);
      int64_t n = sequence_units(a, r, lane);
      const int pairs = __reduce_add_sync(0xFFFFFFFFu, (r.lq + span - 1) / span);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, d);
      if (lane == 0) chunks[ch] = Units{n, pairs};
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
  int32_t never = 0;
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if constexpr (LOAD) return mbar_wait_warp_inline(b, parity, ab);
    else return mbar_wait_warp(b, parity, ab);
  };
  auto take_out = [&](int kb) {  // (rare)
    atomicMin(&taken[0], kb);
    atomicMax(&taken[1], kb);
  };
  // Two warps (lt: the thread among them) bring the codes of K (op 0) or V (op 1) of block g, at positions from kb on, to fp16
  // (exactly) in the block's slot, which is free, and the rows' scales beside them.
  [[maybe_unused]] auto bring_codes = [&](int lt, int op, int g, int slot, int kb, int last, bool edge) {
    if constexpr (Q8) {
      constexpr int PPR = HD / 16, RSTEP = 64 / PPR, NR = kKeys / RSTEP, R = L::kRaw;  // 16-byte pieces of a row; rows of this thread
      const int q = lt >> 5, n_raw = 2 * g + op, rs = n_raw % R;
      // (head_dim 128: half a row of an even and of an odd position to every 8 lanes, so that their stores meet in no bank)
      const int piece = HD == 128 ? ((lane >> 3) & 1) * 4 + (lane & 3) : lane & 3;
      const int row0 = HD == 128 ? q * 4 + (lane >> 4) * 2 + ((lane >> 2) & 1) : q * 8 + (lane >> 2);
      if (!wait(&rawfull[rs], (n_raw / R) & 1)) return false;
      uint4 c[NR];
      const uint32_t raw = smem_u32(smem + L::kRawAt) + rs * L::kRawBytes + row0 * HD + piece * 16;
#pragma unroll
      for (int n = 0; n < NR; ++n)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(c[n].x), "=r"(c[n].y), "=r"(c[n].z), "=r"(c[n].w)
                     : "r"(raw + n * RSTEP * HD));
      float sc = reinterpret_cast<const volatile float*>(smem + L::kRawAt + rs * L::kRawBytes + kKeys * HD)[lt];
      const uint64_t out = *reinterpret_cast<volatile uint64_t*>(&rawhole[rs]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&rawempty[rs]);
      if (edge) {  // values that are not numbers must not meet weights of zero; behind the last row lies anything
        if (kb + lt > last) sc = 0.0f;
        bool some = false;
        if (op == 1) {
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            uint32_t* u = reinterpret_cast<uint32_t*>(&c[n]);
            uint32_t nan = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) nan |= (u[e] & 0x7F7F7F7Fu) + 0x01010101u;
            if (nan & 0x80808080u) {
              some |= kb + row0 + n * RSTEP <= last;
#pragma unroll
              for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int k = 0; k < 32; k += 8)
                  if (((u[e] >> k) & 0x7Fu) == 0x7Fu) u[e] &= ~(0xFFu << k);
            }
          }
          if (!isfinite(sc)) sc = 0.0f, some = true;
        }
        if (some) take_out(kb);
      }
      const uint32_t to = smem_u32(ring) + slot * L::kPair + op * L::kTile + (2 * piece / 8) * L::kBlock + row0 * 128;
      const uint32_t to0 = to + (((2 * piece & 7) ^ (row0 & 7)) << 4), to1 = to + (((2 * piece + 1 & 7) ^ (row0 & 7)) << 4);
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        uint32_t f[8];
        e4m3x4_to_f16(c[n].x, f[0], f[1]);
        e4m3x4_to_f16(c[n].y, f[2], f[3]);
        e4m3x4_to_f16(c[n].z, f[4], f[5]);
        e4m3x4_to_f16(c[n].w, f[6], f[7]);
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to0 + n * RSTEP * 128), "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3]) : "memory");
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to1 + n * RSTEP * 128), "r"(f[4]), "r"(f[5]), "r"(f[6]), "r"(f[7]) : "memory");
      }
      SlotScales& z = s_scale[slot];
      if (op == 0) {
        z.k[lt] = sc;
        if (lt == 0) hole[slot] = out;
      } else {
        const float lv = log2_scale_of(sc);
        z.v[lt] = sc;
        z.lv[lt] = lv;
        float top = lv;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        if (lane == 0) z.top[q] = top;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(op ? &vfull[slot] : &full[slot]);
    }
    return true;
  };

  if (warp >= 8 && warp < 12) {
    if constexpr (LOAD) give_registers<kIssueRegs>();
    if (warp == 10) {
      // ---- finds the pieces of work of this CTA's range and asks for their queries
      Finder f(a, lane);
      const int hkv = a.c.n_kv_heads;
      int64_t head_units = 0;  // of one KV head's line
      int32_t pairs = 0;
      if (n_chunks == 1) {
        f.hold(0, a.status);
        f.add_up();
        head_units = __shfl_sync(0xFFFFFFFFu, f.upto, 31);
        pairs = __reduce_add_sync(0xFFFFFFFFu, f.pairs());
      } else {
        for (int ch = lane; ch < n_chunks; ch += 32) head_units += chunks[ch].units, pairs += chunks[ch].pairs;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) head_units += __shfl_xor_sync(0xFFFFFFFFu, head_units, d);
        pairs = __reduce_add_sync(0xFFFFFFFFu, pairs);
      }
      const int parts = chunk_parts(head_units * hkv, (int64_t)pairs * hkv, gridDim.x);
      // the cut in front of CTA c: hkv x head_units x c / parts units from the line's start
      auto cut_at = [&](int c) {
        if (c >= parts) return Place{hkv, 0, 0, 0};
        const int h = hkv * c / parts;
        int64_t x = (int64_t)((uint64_t)head_units * (uint32_t)(hkv * c - h * parts) / (uint32_t)parts);
        int ch = 0;
        if (n_chunks > 1) {
          for (; ch + 1 < n_chunks; ch += 32) {  // 32 chunks at a time
            const int64_t n = ch + lane < n_chunks ? chunks[ch + lane].units : 0, sum = scan_inclusive(n, lane);
            const int k = __popc(__ballot_sync(0xFFFFFFFFu, sum <= x));
            if (k < 32) {
              x -= __shfl_sync(0xFFFFFFFFu, sum - n, k);
              ch += k;
              break;
            }
            x -= __shfl_sync(0xFFFFFFFFu, sum, 31);
          }
          ch = min(ch, n_chunks - 1);
          f.hold(ch, nullptr);
          f.add_up();
        }
        return f.place(h, x);
      };
      const Place end = cut_at(range + 1);
      Place p = cut_at(range);
      fence_async_smem();  // (the sums have been read before copies take their place)
      if (a.part_state && lane == 0 && !(p.before(end) && p.j > 0 && head_units > 0)) say_part(a, range, kPartNone);
      int published = 0, nq = 0;
      bool ok = true;
      Rows r = shfl_rows(f.mine, p.b & 31);
      pairs = (r.lq + span - 1) / span;
      while (ok && head_units > 0 && p.before(end)) {
        if (p.t >= pairs) {  // the next sequence with rows, or the next head
          p.t = p.j = 0;
          int b = p.b + 1;
          while (true) {
            if (b >= a.c.n_seqs) {
              b = 0;
              if (++p.h >= hkv) break;
            }
            f.hold(b >> 5, nullptr);
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, f.mine.lq > 0) >> (b & 31);
            if (m) {
              b += __ffs(m) - 1;
              break;
            }
            b = (b | 31) + 1;
          }
          p.b = b;
          r = shfl_rows(f.mine, p.b & 31);
          pairs = (r.lq + span - 1) / span;
          continue;
        }
        const int n = pair_blocks(a, r, p.t);
        const bool here = p.h == end.h && p.b == end.b && p.t == end.t;
        const int i1 = here ? min(end.j, n) : n;
        if (p.j < i1 || n == 0) {
          const int s = published % kItems;
          if (published >= kItems && !(ok = wait(&iempty[s], (published / kItems - 1) & 1))) break;
          const bool before = p.j > 0, behind = i1 < n;
          const Item w{r.q0, r.lq, r.len, p.b, p.t * span, p.h, p.j, i1, before ? 0 : behind ? 1 : -1, 0};
          __syncwarp();
          if (lane == 0) {
            items[s] = w;
            mbar_arrive(&ifull[s]);
          }
          ++published;
          if (i1 > p.j) {
            if (nq > 0 && !(ok = wait(qempty, (nq - 1) & 1))) break;
            if (lane == 0) {
              const int boxes = w.half(a.tok) ? 1 : 2;
              mbar_arrive_expect_tx(qfull, (uint32_t)(boxes * a.tok * a.group) * 128 * (HD / 64));
              for (int t = 0; t < boxes; ++t)
                for (int c = 0; c < HD / 64; ++c)
                  tma_load_3d(Qs + t * L::kQTile + c * L::kQBlock, &mq, c * 64, w.h * a.group, w.q0 + w.t0 + t * a.tok, qfull);
            }
            ++nq;
            __syncwarp();
          }
        }
        p.j = 0;
        ++p.t;
      }
      if (ok) {
        const int s = published % kItems;
        ok = published < kItems || wait(&iempty[s], (published / kItems - 1) & 1);
        if (ok && lane == 0) {
          items[s].stop = 1;
          mbar_arrive(&ifull[s]);
        }
      }
      if (!ok) *ab = 1;
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
          if (!(ok = wait(&ifull[is], (it / kItems) & 1))) break;
          const Item w = items[is];
          __syncwarp();
          if (lane == 0) mbar_arrive(&iempty[is]);
          if (w.stop) break;
          const int last = w.last(span);
          const ChunkSpan sp = chunk_span(w.first(), last, a.window, a.sinks);
          const int32_t* trow = a.c.table + (int64_t)w.b * a.c.table_width;
          int next = w.i0 < w.i1 ? table_entry(a, trow, chunk_block(sp, w.i0) * kKeys + bi * box) : 0;
          for (int i = w.i0; i < w.i1; ++i) {
            const int pos = chunk_block(sp, i) * kKeys + bi * box, s = g % NS;
            const int page = page_of(a, next, pos, box, sp.low, last);
            if (i + 1 < w.i1) next = table_entry(a, trow, chunk_block(sp, i + 1) * kKeys + bi * box);
            if (g >= NS && !(ok = wait(&empty[s], (g / NS - 1) & 1))) break;
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
      } else if constexpr (Q8) {
        // ---- copies blocks of codes with their scales: the rows of a page and head are consecutive.  All of a block's copies go out
        // at once, a lane's each: of a page K's codes, V's, K's scales and V's.  (This warp's instructions count: with K's and V's copies
        // one after the other, 4 rows of each of 32 sequences over 8,192 positions in pages of 16 took 295 us, this way 255.)
        constexpr int R = L::kRaw;
        const int lg = min(a.c.log2_page, 6), box = 1 << lg, in_page = (1 << a.c.log2_page) - 1;
        const bool is_v = lane & 1, is_scale = lane & 2;
        const uint8_t* const base = is_scale ? reinterpret_cast<const uint8_t*>(is_v ? a.c.v_scale : a.c.k_scale) : is_v ? a.c.v : a.c.k;
        const int64_t page_step = is_scale ? a.c.scale_stride * 4 : a.c.page_bytes;
        const uint32_t row_bytes = is_scale ? 4 : HD, bytes = box * row_bytes;
        const uint32_t raw = smem_u32(smem + L::kRawAt) + (is_scale ? kKeys * HD : 0);
        const bool on = !is_scale || a.even_scales;
        const uint32_t expect = kKeys * HD + (a.even_scales ? kKeys * 4 : 0);
        uint32_t s = is_v, phase = 1;  // this lane's buffer, of the block's K or V
        int g = 0;                     // blocks so far
        bool ok = true;
        for (int it = 0; ok; ++it) {
          const int is = it % kItems;
          if (!(ok = wait(&ifull[is], (it / kItems) & 1))) break;
          const Item w = items[is];
          __syncwarp();
          if (lane == 0) mbar_arrive(&iempty[is]);
          if (w.stop) break;
          const int last = w.last(span);
          const ChunkSpan sp = chunk_span(w.first(), last, a.window, a.sinks);
          const int32_t* trow = a.c.table + (int64_t)w.b * a.c.table_width;
          const uint8_t* const head = base + (int64_t)(w.h << a.c.log2_page) * row_bytes;
          const int mine = (lane >> 2) << lg;  // this lane's first position of a block
          int next = w.i0 < w.i1 ? table_entry(a, trow, chunk_block(sp, w.i0) * kKeys + mine) : 0;
          for (int i = w.i0; i < w.i1; ++i, ++g) {
            const int kb = chunk_block(sp, i) * kKeys;
            int entry = next;
            if (i + 1 < w.i1) next = table_entry(a, trow, chunk_block(sp, i + 1) * kKeys + mine);
            if (!(ok = wait(&rawempty[s], phase))) break;
            uint64_t out = 0;  // positions without a place
#pragma unroll 1
            for (int at = mine; at - mine < kKeys; at += 8 << lg) {  // (more than once where a page has less than 8 positions)
              const int pos = kb + at;
              if (at != mine) entry = table_entry(a, trow, pos);
              const int page = at < kKeys ? page_of(a, entry, pos, box, sp.low, last) : -2;
              for (uint32_t m = __ballot_sync(0xFFFFFFFFu, page == -1); m; m &= m - 1)
                out |= (box == 64 ? ~0ull : (1ull << box) - 1) << __shfl_sync(0xFFFFFFFFu, at, __ffs(m) - 1);
              if (on && at < kKeys)
                bulk_load(raw + s * L::kRawBytes + at * row_bytes,
                          page < 0 ? reinterpret_cast<const uint8_t*>(zero_codes) : head + page * page_step + (pos & in_page) * row_bytes,
                          bytes, &rawfull[s]);
            }
            if (!a.even_scales) {
              const uint32_t sk = __shfl_sync(0xFFFFFFFFu, s, 0), sv = __shfl_sync(0xFFFFFFFFu, s, 1);
#pragma unroll 1
              for (int x = lane; x < 2 * kKeys; x += 32) {
                const int r = x % kKeys, pos = kb + r, e = page_of(a, table_entry(a, trow, pos), pos, 1, sp.low, last);
                const float* const scales = x < kKeys ? a.c.k_scale : a.c.v_scale;
                reinterpret_cast<float*>(smem + L::kRawAt + (x < kKeys ? sk : sv) * L::kRawBytes + kKeys * HD)[r] =
                    e < 0 ? 0.0f : scales[(int64_t)e * a.c.scale_stride + (w.h << a.c.log2_page) + (pos & in_page)];
              }
              __syncwarp();
            }
            if (lane < 2) {  // (K's buffer and V's; behind the copies, whose bytes count all the same)
              rawhole[s] = out;
              mbar_arrive_expect_tx(&rawfull[s], expect);
            }
            if (out && lane == 0) {
              *holes = 1;
              report(a.status, ADP_ERR_INVALID_ARG);
            }
            s += 2;
            if (s >= R) s -= R, phase ^= 1;
          }
        }
        if (!ok) *ab = 1;
        if (lane == 0)
          for (int i = 2 * g > R ? 2 * g - R : 0; i < 2 * g; ++i) mbar_wait(&rawfull[i % R], (i / R) & 1, &never, a.wait_ns);
        __syncwarp();
      }
    } else {
      // ---- warps 9 and 11 issue the MMAs of tile A and of tile B
      constexpr uint32_t id_s0 = tc_idesc_f16(BF, 128, kKeys);
      constexpr uint32_t id_o = tc_idesc_f16(BF, 128, HD) | kTcIdescBMn;
      constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);
      const uint32_t id_s = id_s0 | a.neg;
      const uint32_t t = warp == 11;
      const uint32_t q_lo0 = (smem_u32(Qs) >> 4) | (1u << 16);
      const uint32_t k_lo = (smem_u32(ring) >> 4) | (1u << 16);
      const uint32_t v_lo = ((smem_u32(ring) + L::kTile) >> 4) | ((L::kBlock >> 4) << 16);
      const uint32_t tS = tmem + t * 128, tO = tmem + 256 + t * 128;
      uint32_t ks = 0, kphase = 0, vs = 0, vphase = 0;  // the ring's next block, and the next own block to weigh
      uint32_t s_buf = 0, s_phase = 0, p_buf = 0, p_phase = 0, q_phase = 0;
      bool ok = true;
#pragma unroll 1
      for (int it = 0; ok; ++it) {
        const int is = it % kItems;
        if (!(ok = wait(&ifull[is], (it / kItems) & 1))) break;
        const Item w = items[is];
        __syncwarp();
        if (elect_one()) mbar_arrive(&iempty[is]);
        __syncwarp();
        if (w.stop) break;
        const int n = w.i1 - w.i0;
        if (n == 0) continue;
        const Own own = own_blocks(w, chunk_span(w.first(), w.last(span), a.window, a.sinks), t, a.tok);
        const uint32_t q_lo = q_lo0 + (w.half(a.tok) ? 0 : t * (L::kQTile >> 4));
        if (!(ok = wait(QCONV ? qready : qfull, q_phase))) break;
        q_phase ^= 1;
        int at = 0;  // blocks of the item that have been waited for
        vs = ks + own.off;
        vphase = kphase;
        if (vs >= NS) vs -= NS, vphase ^= 1;
        // the next block of the item is not this tile's: it is freed once it is there
        auto skip = [&]() {
          if (!wait(&full[ks], kphase)) return false;
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
          if (!wait(&full[ks], kphase) || !wait(&odone[2 * t + s_buf], s_phase ^ 1)) return false;
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
        if (own.n == 0) {
          if (elect_one()) mbar_arrive(qempty);
          __syncwarp();
        }
        // The next block's scores go in front of this one's product.  Where tiles take turns, and with the few slots of fp16 from
        // codes, only if its K is there: the slot that it waits for may be this block's.
        const bool always = !Q8 && own.step == 1;
        int scored = 0;
#pragma unroll 1
        for (int k = 0; k < own.n; ++k) {
          if (scored == k && !(ok = score(scored++))) break;
          if (scored < own.n) {
            bool there = always || __all_sync(0xFFFFFFFFu, mbar_test_wait(&full[ks], kphase));
            while (there && at < own.off + scored * own.step) {
              skip();
              there = __all_sync(0xFFFFFFFFu, mbar_test_wait(&full[ks], kphase));
            }
            if (there && !(ok = score(scored++))) break;
          }
          if (!(ok = wait(&pready[2 * t + p_buf], p_phase))) break;
          if constexpr (Q8) {
            if (!(ok = wait(&vfull[vs], vphase))) break;
          }
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
          if (vs >= NS) vs -= NS, vphase ^= 1;
        }
        while (ok && at < n) ok = skip();
      }
      if (!ok) *ab = 1;
      if (elect_one()) tc_commit(done);  // on every path: arrives once no MMA of this warp is in flight
      __syncwarp();
    }
  } else if (warp >= 12) {
    if constexpr (LOAD) {
      give_registers<kLoadRegs>();
      const int lt = threadIdx.x - 384;
      bool ok = true;
      auto wait_slot = [&](int n) { return n < NS || wait(&empty[n % NS], (n / NS - 1) & 1); };
      if constexpr (Q8) {
        // ---- two warps bring codes of K to fp16 in the ring, and two those of V (all four K's, then V's: 236 us for 4 rows of each of
        // 32 sequences over 8,192 positions in pages of 64, this way 206)
        int g = 0, slot = 0;  // blocks so far, and the next one's slot
        for (int it = 0; ok; ++it) {
          const int is = it % kItems;
          if (!(ok = wait(&ifull[is], (it / kItems) & 1))) break;
          const Item w = items[is];
          __syncwarp();
          if (lane == 0) mbar_arrive(&iempty[is]);
          if (w.stop) break;
          const int first = w.first(), last = w.last(span);
          const ChunkSpan sp = chunk_span(first, last, a.window, a.sinks);
          for (int i = w.i0; ok && i < w.i1; ++i, ++g) {
            const int kb = chunk_block(sp, i) * kKeys;
            const bool edge = edge_block(kb, first, last, a.window, a.sinks);
            ok = wait_slot(g) && bring_codes(lt & 63, lt >> 6, g, slot, kb, last, edge);
            if (++slot == NS) slot = 0;
          }
        }
      } else {
        // ---- four warps that copy rows of 16-bit pages too small for tensor copies: consecutive lanes take consecutive
        // 16-byte pieces of a row
        constexpr int PPR = HD / 8, RSTEP = 128 / PPR, NR = kKeys / RSTEP, kAhead = NS >= 5 ? 2 : 1;
        // block g waits for the slot of block g - NS, whose product is issued behind the scores of its tile's next block
        // (g - NS + 2 where tiles take turns): those under way must all lie behind that one
        static_assert(kAhead <= NS - 3, "");
        const int piece = lt % PPR, row0 = lt / PPR;
        int g = 0, landed = 0;  // blocks asked for, and those handed over
        uint32_t gaps = 0;      // of the blocks under way, the last one lowest: this thread's row has no place
        // positions of a block without a place, said by the warps that hold its rows
        auto say_holes = [&](int s, bool gap) {
          if (warp >= 14) return;
          const uint32_t m = __ballot_sync(0xFFFFFFFFu, gap);
          if (lane == 0) {
            reinterpret_cast<uint32_t*>(&hole[s])[warp - 12] = m;
            if (m) {
              *holes = 1;
              report(a.status, ADP_ERR_INVALID_ARG);
            }
          }
        };
        auto hand_over = [&]() {  // the oldest block under way: its copies have ended for this thread
          const int s = landed % NS;
          say_holes(s, (gaps >> (g - 1 - landed)) & 1);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[s]);
          ++landed;
        };
        auto flush = [&]() {
          cp_async_wait<0>();
          while (landed < g) hand_over();
        };
        for (int it = 0; ok; ++it) {
          const int is = it % kItems;
          // (a piece of work that is not known yet may wait for the blocks under way)
          if (!__all_sync(0xFFFFFFFFu, mbar_test_wait(&ifull[is], (it / kItems) & 1))) {
            flush();
            if (!(ok = wait(&ifull[is], (it / kItems) & 1))) break;
          }
          const Item w = items[is];
          __syncwarp();
          if (lane == 0) mbar_arrive(&iempty[is]);
          if (w.stop) break;
          const int last = w.last(span), in_page = (1 << a.c.log2_page) - 1;
          const ChunkSpan sp = chunk_span(w.first(), last, a.window, a.sinks);
          const int32_t* trow = a.c.table + (int64_t)w.b * a.c.table_width;
          int next[NR], next_own = 0;
          auto look_up = [&](int i) {
            const int kb = chunk_block(sp, i) * kKeys;
#pragma unroll
            for (int n = 0; n < NR; ++n) next[n] = table_entry(a, trow, kb + row0 + n * RSTEP);
            next_own = table_entry(a, trow, kb + (lt & (kKeys - 1)));
          };
          if (w.i0 < w.i1) look_up(w.i0);
          for (int i = w.i0; i < w.i1; ++i) {
            const int kb = chunk_block(sp, i) * kKeys;
            int page[NR];
#pragma unroll
            for (int n = 0; n < NR; ++n) page[n] = page_of(a, next[n], kb + row0 + n * RSTEP, 1, sp.low, last);
            gaps = (gaps << 1) | (page_of(a, next_own, kb + (lt & (kKeys - 1)), 1, sp.low, last) == -1 ? 1u : 0u);
            if (i + 1 < w.i1) look_up(i + 1);
            if (!(ok = wait_slot(g))) break;
#pragma unroll
            for (int n = 0; n < 2 * NR; ++n) {
              const int row = row0 + (n % NR) * RSTEP, pg = page[n % NR];
              const int64_t cell = (int64_t)max(pg, 0) * a.c.page_bytes +
                                   (int64_t)((w.h << a.c.log2_page) + ((kb + row) & in_page)) * (HD * 2) + piece * 16;
              cp_async16(smem_u32(ring + (g % NS) * L::kPair) + (n >= NR ? L::kTile : 0) + (piece >> 3) * L::kBlock + row * 128 +
                             (((piece & 7) ^ (row & 7)) << 4),
                         (n >= NR ? a.c.v : a.c.k) + cell, pg >= 0);
            }
            cp_async_commit();
            ++g;
            if (g - landed > kAhead) {
              cp_async_wait<kAhead>();
              hand_over();
            }
          }
        }
        flush();
      }
      if (!ok) *ab = 1;
    }
  } else {
    // ---- softmax: warps 0-3 tile A, 4-7 tile B; thread = row = TMEM lane
    if constexpr (LOAD) take_registers<kSoftmaxRegs>();
    const int t = warp >> 2, r = threadIdx.x & 127, sub = warp & 3;
    const uint32_t lanes = (uint32_t)(sub * 32) << 16;
    const uint32_t tS = tmem + lanes + t * 128, tO = tmem + lanes + 256 + t * 128;
    bool ok = true;
    uint32_t ns = 0, nj = 0, nq = 0;  // own blocks, meetings of the softmax warps, items with queries so far
    uint32_t g = 0;                   // ring blocks of the items before
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(joined);
      return wait(joined, nj++ & 1);
    };
    for (int it = 0; ok; ++it) {
      const int is = it % kItems;
      if (!(ok = wait(&ifull[is], (it / kItems) & 1))) break;
      const Item w = items[is];
      if (w.stop) break;
      const int first = w.first(), last = w.last(span), n = w.i1 - w.i0;
      const ChunkSpan sp = chunk_span(first, last, a.window, a.sinks);
      const Own own = own_blocks(w, sp, t, a.tok);
      const bool half = w.half(a.tok);
      const int row_tok = r / a.group, row_head = r - row_tok * a.group;
      const int tok = w.t0 + (half ? 0 : t * a.tok) + row_tok;
      const bool live = row_tok < a.tok && tok < w.lq;
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
          if (!(ok = wait(qfull, nq & 1))) break;
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
            if (row_tok < a.tok) {
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
          if (!(ok = wait(qready, nq & 1))) break;
          // (kept finite, as the scale itself)
          scale = fminf(fmaxf(scale * s_qf[half ? r : t * kRows + r], kScaleMin), 3.40282347e38f);
          ++nq;
        }
      }
      // the running maximum (and ms, what is subtracted from scores) and sum, and the score above which the maximum is
      // replaced (never by what stands in rows that are not the sequence's: it must not decide how the others are rounded)
      float m = -INFINITY, ms = 0.0f, l = 0.0f, limit = live ? -INFINITY : INFINITY;
      // e4m3: what weighs V's codes are the products weight x value scale, which have a running maximum of their own, mo
      // (base-2 exponents: score + log2 of the scale); O is relative to it, and vc = 2^((m - mo) / 2), twice, brings them there
      float mo = -INFINITY, vc = 1.0f;
      // The softmax of own block k, whose scores lie in buffer buf: P takes their place, 16 bits each.
      auto block = [&](int k, uint32_t buf, int slot, int kb) {
        constexpr int N = kKeys;
        float x[N];
        tmem_ld64(tS + buf * 64, x);
        [[maybe_unused]] const SlotScales& z = s_scale[Q8 ? slot : 0];
        if constexpr (Q8) {
#pragma unroll
          for (int c = 0; c < N; c += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&z.k[c]);
            const float2 u = __fmul2_rn(make_float2(x[c], x[c + 1]), make_float2(f.x, f.y));
            const float2 v = __fmul2_rn(make_float2(x[c + 2], x[c + 3]), make_float2(f.z, f.w));
            x[c] = u.x, x[c + 1] = u.y, x[c + 2] = v.x, x[c + 3] = v.y;
          }
        }
        const bool hidden = kb + N - 1 > warp_first || (kb <= warp_last - a.window && kb + N - 1 >= a.sinks);
        if (hidden || *holes) {
          // columns up to this row's position, from its window's first on or of the first ones, but those without a place
          uint64_t see = below(pos - kb + 1) & (~below(from - kb) | below(a.sinks - kb));
          if (*holes) see &= ~*reinterpret_cast<volatile uint64_t*>(&hole[slot]);
          const uint32_t lo = (uint32_t)see, hi = (uint32_t)(see >> 32);
#pragma unroll
          for (int c = 0; c < N; ++c) x[c] = ((c < 32 ? lo : hi) >> (c & 31)) & 1 ? x[c] : -INFINITY;
        }
        float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < N - 4; c += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) top[e] = max3(top[e], x[c + e], x[c + 4 + e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], x[N - 4 + e]);
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
            for (int c = 0; c < N; c += 4) {
              const float4 lv = *reinterpret_cast<const float4*>(&z.lv[c]);
              mw = fmaxf(fmaxf(mw, fmaf(x[c], scale, lv.x)), fmaf(x[c + 1], scale, lv.y));
              mw = fmaxf(fmaxf(mw, fmaf(x[c + 2], scale, lv.z)), fmaf(x[c + 3], scale, lv.w));
            }
            mw = live ? fmaxf(mo, mw) : mo;
            f = mw == -INFINITY ? 1.0f : exp2_fast(mo - mw);
            mo = mw;
            vc = mw == -INFINITY ? 1.0f : exp2_fast(0.5f * (m - mw));
          }
          if (k > 0) {
            // own block k - 1's product must be in O
            if (!wait(&odone[2 * t + (buf ^ 1)], ((ns - 1) >> 1) & 1)) return false;
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
        [[maybe_unused]] const float2 vc2 = make_float2(vc, vc);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int c0 = 0; c0 < N; c0 += 32) {
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            [[maybe_unused]] float4 f;
            if constexpr (Q8) f = *reinterpret_cast<const float4*>(&z.v[c0 + e]);
#pragma unroll
            for (int d = 0; d < 4; d += 2) {
              const float2 y = __ffma2_rn(make_float2(x[c0 + e + d], x[c0 + e + d + 1]), sc, nm);
              float2 p = make_float2(exp2_fast(y.x), exp2_fast(y.y));  // (0 where x is -infinity: not seen)
              sum[d >> 1] = __fadd2_rn(sum[d >> 1], p);
              if constexpr (Q8)  // (in this order nothing that counts leaves fp32's range)
                p = __fmul2_rn(__fmul2_rn(__fmul2_rn(p, vc2), d ? make_float2(f.z, f.w) : make_float2(f.x, f.y)), vc2);
              u[(e + d) >> 1] = pack2(p.x, p.y, BF ? DT_BF16 : DT_F16);
            }
          }
          tmem_st16(tS + buf * 64 + c0 / 2, u);
        }
        tmem_st_wait();
        tc_fence_before();
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        return true;
      };
      for (int k = 0; k < own.n; ++k, ++ns) {
        const uint32_t buf = ns & 1;
        const int i = own.off + k * own.step, slot = (g + i) % NS, kb = chunk_block(sp, w.i0 + i) * kKeys;
        if (!(ok = wait(&sfull[2 * t + buf], (ns >> 1) & 1))) break;
        tc_fence_after();
        __syncwarp();
        if constexpr (Q8) {  // (the scales of V come with V)
          if (!(ok = wait(&vfull[slot], ((g + i) / NS) & 1))) break;
        }
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
              take_out(kb);
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
          ok = block(k, buf, slot, kb);
          if (!ok) break;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[2 * t + buf]);
      }
      // ---- behind the last two products (the others' ends were waited for when S took their P's place)
      if (ok && own.n > 1) ok = wait(&odone[2 * t + (ns & 1)], ((ns - 2) >> 1) & 1);
      if (ok && own.n > 0) ok = wait(&odone[2 * t + (~ns & 1)], ((ns - 1) >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      g += n;
      // (e4m3: O is relative to mo, and brought to m in two steps)
      float own_f = Q8 && mo > -INFINITY ? exp2_fast(0.5f * (mo - m)) : 1.0f;
      auto load_o = [&](int c0, float f, float (&o)[16]) {  // 16 columns of O times f, 0 where nothing was seen
        uint32_t u[16];
        tmem_ld16(tO + c0, u);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float y = __uint_as_float(u[e]);
          if (Q8) y = y * own_f * own_f;
          o[e] = l == 0.0f ? 0.0f : y * f;
        }
      };
      uint8_t* const out = a.out + (int64_t)(w.q0 + tok) * a.out_stride + (int64_t)(w.h * a.group + row_head) * HD * 2;
      const int64_t prow = (int64_t)range * a.rows_cap;  // the first row of this range's partial result
      const bool says = !half || t == 0;  // of the warps with these rows, the one that speaks for them
      if (w.part == 1 && warp_live) {
        // ---- the first part of several: the others' results, of the next ranges, come to its accumulators; warps that have the
        // same rows take turns at them (8 rows over 16,000 positions, 19 parts a KV head: 43 us, 61 with one warp)
        const int turns = half ? 2 : 1, own_turn = half ? t : 0;
        int n_parts = 0;
        bool more = true;
        for (int c0 = range + 1; more && c0 < (int)gridDim.x; c0 += 32) {  // a lane for every range
          const uint64_t t0 = globaltimer();
          uint32_t those;
          while (true) {
            const int32_t state = c0 + lane < (int)gridDim.x ? part_said(a, c0 + lane) : kPartNone;
            const uint32_t ends = __ballot_sync(0xFFFFFFFFu, state == kPartEnds), open = __ballot_sync(0xFFFFFFFFu, state == kPartOpen);
            const uint32_t mine = ends ^ (ends - 1);  // up to the first end, or all of them
            those = __ballot_sync(0xFFFFFFFFu, state == kPartEnds || state == kPartGoesOn) & mine;
            more = ends == 0;
            if (!(open & mine)) break;
            if (!(ok = __all_sync(0xFFFFFFFFu, *ab == 0 && globaltimer() - t0 <= a.wait_ns))) break;
          }
          __syncwarp();
          if (!ok) break;
          for (; those; those &= those - 1) {
            if (n_parts++ % turns != own_turn) continue;
            const int c = c0 + __ffs(those) - 1;
            const int64_t base = (int64_t)c * a.rows_cap + (half ? 0 : t * kRows) + sub * 32;
            const float2 ml = live ? a.part_ml[base + lane] : make_float2(-INFINITY, 0.0f);
            const float4* from = reinterpret_cast<const float4*>(a.part_o) + base * (HD / 4) + lane;
            const float mn = fmaxf(m, ml.x), to = mn == -INFINITY ? 0.0f : mn;
            const float f = exp2_fast(m - to), g = exp2_fast(ml.x - to);
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 64) {
              float4 x[16];
#pragma unroll
              for (int p = 0; p < 16; ++p) x[p] = live ? from[(c0 / 4 + p) * 32] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                float o[16];
                load_o(c0 + 16 * h, f, o);
                uint32_t u[16];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                  const float4 y = x[4 * h + p];
                  u[4 * p] = __float_as_uint(fmaf(y.x, g, o[4 * p])), u[4 * p + 1] = __float_as_uint(fmaf(y.y, g, o[4 * p + 1]));
                  u[4 * p + 2] = __float_as_uint(fmaf(y.z, g, o[4 * p + 2])), u[4 * p + 3] = __float_as_uint(fmaf(y.w, g, o[4 * p + 3]));
                }
                tmem_st16(tO + c0 + 16 * h, u);
              }
            }
            tmem_st_wait();
            m = mn;
            l = fmaf(l, f, g * ml.y);
            own_f = 1.0f;  // (O is relative to m now)
          }
        }
        if (!ok) break;
      }
      const bool goes_on = w.i1 < sp.n;
      int lo = 0, hi = -1;  // the blocks that values were taken out of
      auto look = [&]() {
        lo = *reinterpret_cast<volatile int32_t*>(&taken[0]);
        hi = *reinterpret_cast<volatile int32_t*>(&taken[1]);
      };
      uint8_t* const stage = smem + L::kOut;
      if (half) {
        // ---- both tiles (and all their warps) have these rows: maxima and sums, then the results, some columns at a time
        s_half[t * kRows + r] = m;
        s_half[(2 + t) * kRows + r] = l;
        if (!(ok = meet())) break;
        look();
        float top = -INFINITY, total = 0.0f;
        for (int q = r; q < 2 * kRows; q += kRows) top = fmaxf(top, s_half[q]);
        const float base = top == -INFINITY ? 0.0f : top;
        for (int q = r; q < 2 * kRows; q += kRows) total = fmaf(exp2_fast(s_half[q] - base), s_half[2 * kRows + q], total);
        const float f = exp2_fast(m - base) * (w.part == 0 ? 1.0f : total == 0.0f ? 0.0f : 1.0f / total);
        if (w.part == 0 && live && says) a.part_ml[prow + r] = make_float2(top, total);
        // (two buffers of 256 x C floats: of the tiles' rows, up to 32, 64 or 128, and as many times C columns as they leave room for)
        constexpr int C = L::kOutCols, P = C / 4;
        const int fit = min(w.lq - w.t0, a.tok) * a.group, lg = fit > 64 ? 7 : fit > 32 ? 6 : 5;
        auto cell = [&](int b, int q, int p) {
          return reinterpret_cast<float4*>(stage + (b * 2 * kRows + q) * C * 4 + ((p ^ (P == 4 ? (q >> 1) & 3 : (q >> 2) & 1)) << 4));
        };
        // this thread adds up piece p of some columns of some rows
        const int id = t * kRows + r, p = id % P;
        constexpr int kMine = P / 2;
        uint8_t* to[kMine];
        int of[kMine], col_of[kMine], tok_of[kMine];  // the cell of the first summand, the columns' and the row's place
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
          const int x = id / P + 64 * k, q0 = x & ((1 << lg) - 1), set = x >> lg;
          of[k] = q0 < fit ? (set << (lg + 1)) + q0 : -1;
          col_of[k] = set * C + 4 * p;
          tok_of[k] = q0 / a.group;
          to[k] = w.part == 0 ? reinterpret_cast<uint8_t*>(a.part_o) + ((prow + (q0 & ~31)) * (HD / 4) + (q0 & 31)) * 16
                              : a.out + (int64_t)(w.q0 + w.t0 + tok_of[k]) * a.out_stride +
                                    (int64_t)(w.h * a.group + q0 - tok_of[k] * a.group) * HD * 2;
        }
        auto add_up = [&](int b, int k, int col) {
          float4 v = *cell(b, of[k], p), y = *cell(b, of[k] + (1 << lg), p);
          v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
          if (hi >= 0) {
            y = taken_out<HD, CDT>(a, w, w.len - w.lq + w.t0 + tok_of[k], col, lo, hi);
            v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
          }
          if (w.part == 0) *reinterpret_cast<float4*>(to[k] + col * 128) = v;  // (a piece's 32 rows are consecutive there)
          else *reinterpret_cast<uint2*>(to[k] + col * 2) = make_uint2(pack2(v.x, v.y, QDT), pack2(v.z, v.w, QDT));
        };
        int b = 0;
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += C << (7 - lg), b ^= 1) {
          if (warp_live) {
#pragma unroll 1
            for (int set = 0; set < 1 << (7 - lg); ++set) {
              const int c = c0 + set * C;
              float o[16];  // (8 of them where C is 8)
              load_o(c & ~15, f, o);
#pragma unroll
              for (int e = 0; e < P; ++e) {
                float4 v = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                if (C == 8 && (c & 8)) v = make_float4(o[4 * e + 8], o[4 * e + 9], o[4 * e + 10], o[4 * e + 11]);
                *cell(b, (set << (lg + 1)) + (t << lg) + r, e) = v;
              }
            }
          }
          if (!(ok = meet())) break;
#pragma unroll
          for (int k = 0; k < kMine; ++k)
            if (of[k] >= 0) add_up(b, k, c0 + col_of[k]);
        }
        if (w.part == 0) __threadfence();
        if (ok) ok = meet();  // (what comes next takes these maxima, sums and results' place)
        if (!ok) break;
        if (w.part == 0 && threadIdx.x == 0) say_part(a, range, goes_on ? kPartGoesOn : kPartEnds);
      } else if (w.part == 0) {
        // ---- a part: consecutive lanes' rows are consecutive there
        look();
        if (live) a.part_ml[prow + t * kRows + r] = make_float2(m, l);
        if (warp_live) {
          float4* const to = reinterpret_cast<float4*>(a.part_o) + (prow + t * kRows + sub * 32) * (HD / 4) + lane;
#pragma unroll 1
          for (int c0 = 0; c0 < HD; c0 += 16) {
            float o[16];
            load_o(c0, 1.0f, o);
            if (live) {
#pragma unroll
              for (int p = 0; p < 4; ++p) {
                float4 v = make_float4(o[4 * p], o[4 * p + 1], o[4 * p + 2], o[4 * p + 3]);
                if (hi >= 0) {
                  const float4 x = taken_out<HD, CDT>(a, w, pos, c0 + 4 * p, lo, hi);
                  v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
                }
                to[(c0 / 4 + p) * 32] = v;
              }
            }
            __syncwarp();
          }
        }
        __threadfence();
        if (!(ok = meet())) break;
        if (threadIdx.x == 0) say_part(a, range, goes_on ? kPartGoesOn : kPartEnds);
      } else if (warp_live) {
        // ---- whole: this warp's rows go through shared memory, 16-byte pieces swizzled, so that consecutive lanes store
        // consecutive pieces of a row
        constexpr int OB = L::kOutBytes, PP = OB / 16;  // bytes and pieces of a row at a time
        uint8_t* const mine = stage + warp * 32 * OB;
        auto cell = [&](int q, int p) { return reinterpret_cast<uint4*>(mine + q * OB + ((p ^ (PP == 8 ? q & 7 : (q >> 1) & 3)) << 4)); };
        look();
        const uint32_t alive = __ballot_sync(0xFFFFFFFFu, live);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 16) {
          float o[16];
          load_o(c0, inv, o);
          if (hi >= 0 && live) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              const float4 x = taken_out<HD, CDT>(a, w, pos, c0 + 4 * p, lo, hi);
              o[4 * p] += x.x, o[4 * p + 1] += x.y, o[4 * p + 2] += x.z, o[4 * p + 3] += x.w;
            }
          }
          const int at = c0 / 8;  // pieces in front
#pragma unroll
          for (int p = 0; p < 2; ++p)
            *cell(lane, (at + p) % PP) = make_uint4(pack2(o[8 * p], o[8 * p + 1], QDT), pack2(o[8 * p + 2], o[8 * p + 3], QDT),
                                                    pack2(o[8 * p + 4], o[8 * p + 5], QDT), pack2(o[8 * p + 6], o[8 * p + 7], QDT));
          if ((at + 2) % PP) continue;
          __syncwarp();
#pragma unroll
          for (int k = 0; k < PP; ++k) {
            const int q = (k * 32 + lane) / PP;
            uint8_t* to = reinterpret_cast<uint8_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(out), q));
            if ((alive >> q) & 1) *reinterpret_cast<uint4*>(to + (at + 2 - PP + lane % PP) * 16) = *cell(q, lane % PP);
          }
          __syncwarp();
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
  // no MMA may be in flight (nor TMEM in use) when the accumulators are freed
  if (warp == 9) mbar_wait(done, 0, &never, a.wait_ns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
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

// Positions of a page that tensor copies take (32 sequences of up to 8 rows over pages of 8 bf16 positions: 180 us with tensor copies of 8
// rows each, 119 by warps).
constexpr int kMinCopyPage = 16;

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
  p.ctas = chunk_parts(items * (blocks + chunk_over(0, tok)), items, sms);
  if (blocks >= 2 * kChunkMinPart && p.ctas > 1) {
    p.rows_cap = n_rows <= tok ? kRows : 2 * kRows;
    p.bytes = (size_t)p.ctas * (p.rows_cap * ((size_t)kv->head_dim * sizeof(float) + sizeof(float2)) + sizeof(int32_t));
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
  if (a.part_state && (e = cudaMemsetAsync(a.part_state, 0, (size_t)p.ctas * sizeof(int32_t), st)) != cudaSuccess) return e;
  kernel<<<p.ctas, LOAD ? 512 : 384, smem, st>>>(m[0], m[1], m[2], a);
  return cudaGetLastError();
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
  a.even_scales = kv->page_size >= 4 && kv->scale_stride % 4 == 0 && aligned16(kv->k_scale) && aligned16(kv->v_scale);
  a.neg = scale < 0.0f ? kTcIdescANeg : 0;
  a.rows_cap = plan.rows_cap;
  if (plan.bytes) {
    const size_t rows = (size_t)plan.ctas * plan.rows_cap;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + rows * kv->head_dim);
    a.part_state = reinterpret_cast<int32_t*>(a.part_ml + rows);
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
