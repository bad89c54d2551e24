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

constexpr int kRows = 128;            // rows of a query tile (M of the MMA)
constexpr int kKeys = 64;             // keys of a block
constexpr int kThreads = 384;         // 8 softmax warps, one that copies, two that issue MMAs, one that finds the work
constexpr float kRescale = 8.0f;      // base-2 growth of a row's maximum that rescales its output

struct PackedArgs {
  const int32_t* cu_q;
  const int32_t* cu_k;
  const uint8_t* v;
  uint8_t* out;
  int64_t v_stride, out_stride;  // bytes
  int32_t n_seqs, n_q, n_k, hkv, group, tok;
  float scale_log2;              // of |scale|, and above 0
  int32_t* status;
  uint64_t wait_ns;              // limit of every wait
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

// True for one lane of a warp that runs in step, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// The limit of a wait lies 12 bytes behind the abort word in shared memory (8,192 tokens: 0.7% more time than a constant; as an
// argument of every wait 1.1%).
__device__ __forceinline__ uint64_t wait_limit(volatile int32_t* abort) { return *reinterpret_cast<volatile uint64_t*>(abort + 3); }

// A whole warp's wait with one answer for all of it.  What is not over at the first look is waited for in a function of
// its own: between the warps of different roles the instruction caches hold little, and a long wait loop in line cost
// 200 cycles even when there was nothing to wait for.
__device__ __noinline__ bool mbar_wait_warp_slow(uint64_t* b, uint32_t parity, volatile int32_t* abort) {
  const uint64_t t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(b, parity))) return true;
    if ((it & 63) == 0 && __any_sync(0xFFFFFFFFu, *abort != 0 || globaltimer() - t0 > wait_limit(abort))) return false;
  }
}
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* b, uint32_t parity, volatile int32_t* abort) {
  return __all_sync(0xFFFFFFFFu, mbar_try_wait(b, parity)) ? true : mbar_wait_warp_slow(b, parity, abort);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Asks for one CTA of this grid that has not been launched to be taken over: the answer (16 bytes) completes on the
// barrier.
__device__ __forceinline__ void take_over_cta(void* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
// blockIdx.x of the CTA that the answer names, -1 where none was left.
__device__ __forceinline__ int taken_over_cta(const void* answer) {
  uint32_t ok, x;
  asm volatile(
      "{\n .reg .b128 h;\n .reg .pred p;\n ld.shared.b128 h, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n}\n"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return ok ? (int)x : -1;
}

// One CTA's worth of work: 2 x tok tokens from t0 on of one sequence, for one KV head's group of query heads.
struct Item {
  int32_t q0, lq, k0, lk;  // the sequence's first query row, queries, first key row, keys
  int32_t t0, h;
  int32_t stop;            // no work is left
  int32_t pad;
};

// Key blocks that tile t of the item sees: up to those of its last token.
__device__ __forceinline__ int item_blocks(const Item& w, int t, int tok) {
  const int first = w.t0 + t * tok, last = min(first + tok, w.lq) - 1 + w.lk - w.lq;
  return first < w.lq && last >= 0 ? last / kKeys + 1 : 0;
}

// Work item number `index` of all (false: there are fewer): KV head index % hkv of pair index / hkv.  Up to 32
// sequences: pairs in the order of falling cost (key blocks), so that the long ones start first; more: sequence by
// sequence, the last pair (which sees the most keys) first.  A whole warp asks.
__device__ __forceinline__ bool find_item(const PackedArgs& a, int index, int lane, Item* out) {
  const int span = 2 * a.tok;
  int r = index / a.hkv;
  for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
    int q0 = 0, lq = 0, k0 = 0, lk = 0;
    if (b0 + lane < a.n_seqs) {
      packed_range(a.cu_q, b0 + lane, a.n_q, a.status, &q0, &lq);
      packed_range(a.cu_k, b0 + lane, a.n_k, a.status, &k0, &lk);
    }
    const int pairs = (lq + span - 1) / span, all = __reduce_add_sync(0xFFFFFFFFu, pairs);
    if (r >= all) {
      r -= all;
      continue;
    }
    int mine = pairs, skip = 0;  // this lane's pairs of the wanted cost, and those of a higher one
    if (a.n_seqs <= 32) {
      // this lane's pairs that see c key blocks or more
      auto at_least = [&](int c) {
        const int key = (c - 1) * kKeys;  // their last token sees this key
        if (c <= 0) return pairs;
        if (pairs == 0 || lk - 1 < key) return 0;
        const int before = key + 1 - (lk - lq);  // tokens up to the first that sees it
        return pairs - min(before <= span ? 0 : (before + span - 1) / span - 1, pairs - 1);
      };
      int lo = 0, hi = __reduce_max_sync(0xFFFFFFFFu, pairs ? (lk + kKeys - 1) / kKeys : 0) + 1;
      while (hi - lo > 1) {  // the largest cost that more than r pairs reach
        const int mid = (lo + hi) >> 1;
        if ((int)__reduce_add_sync(0xFFFFFFFFu, at_least(mid)) > r) lo = mid; else hi = mid;
      }
      skip = at_least(lo + 1);
      mine = at_least(lo) - skip;
      r -= __reduce_add_sync(0xFFFFFFFFu, skip);
    }
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += o;
    }
    if (r < sum && r >= sum - mine)
      *out = Item{q0, lq, k0, lk, (pairs - 1 - skip - (r - (sum - mine))) * span, index % a.hkv, 0, 0};
    __syncwarp();
    return true;
  }
  return false;
}

template <int HD>
struct PackedSmem {
  static constexpr int kSlots = HD == 128 ? 5 : 8;          // of a block of K and one of V
  static constexpr uint32_t kQBlock = 128 * 128;            // 128 rows x 64 elements, swizzled
  static constexpr uint32_t kQTile = (HD / 64) * kQBlock;
  static constexpr uint32_t kBlock = kKeys * 128;           // the same of K or V
  static constexpr uint32_t kTile = (HD / 64) * kBlock;
  static constexpr uint32_t kPair = 2 * kTile;
  static constexpr uint32_t kBars = 2 * kQTile + kSlots * kPair;  // Q tiles, ring, then the items and the barriers
  static constexpr size_t kBytes = 1024 + kBars + 768;
};

// fp16 weights are held 2^7 times larger (and so is their sum): up to 2^15 beside a maximum that is stale by 2^8, they stay
// below fp16's 65,504, and a weight keeps all its bits down to 2^-21 of the largest and some down to 2^-32, where 2^-14 and
// 2^-25 would let the tail of a long context vanish beside one dominating key.  (bf16 has fp32's range.)
template <bool BF16>
constexpr float kWeightUp = BF16 ? 0.0f : 7.0f;

constexpr int kItems = 2;  // the item worked on and the next one: more known ahead would keep work from idle SMs

// A persistent kernel: a CTA works on items (one KV head's group of query heads for 2 x tok consecutive tokens of one
// sequence) until none is left, starting with its own index and taking over CTAs that have not been launched, so that
// the SMs stay evenly loaded whatever the lengths.  An item is two tiles A and B of 128 rows (row = token x group +
// head: tok = 128 / group tokens, so a group's heads share K and V and the causal edge is only tok tokens wide).
// Three warpgroups: warps 0-3 the softmax of tile A, 4-7 of tile B (thread = row = TMEM lane), warp 8 copies, warps 9 and
// 11 issue the MMAs of tile A and of tile B, warp 10 finds the items.
//  - copies: both Q tiles, and blocks of 64 keys of K and V into a ring of slots (128-byte swizzled), running ahead into
//    the next item;
//  - S = Q K^T per tile and block into one of the tile's two 64-column buffers in TMEM; the softmax reads S, writes P
//    (16-bit) over it, and O += P V takes P from TMEM and V as the MN-major operand.  Block j + 1's scores are issued
//    in front of block j's products, so that the tensor cores have S(j + 1) under way while the softmax works on block j
//    (with one buffer of 128 keys the two took turns: 502 us for 8,192 tokens of 32 / 8 heads).  At an item's end the next
//    one's first scores take their place if its Q is there;
//  - a row's running maximum is replaced only when it grows by more than 2^8 (decided per warp): O and the sum carry the
//    same stale factor, which cancels.
// TMEM: S/P of A and B (2 x 64 columns each), O of A and B (HD columns each).
// Bound by the softmax warps and the MMAs together: 8,192 bf16 tokens of 32 / 8 heads in 368 us (1,490 TFLOP/s; the
// library's GEMM reaches 1,892).
// Keys that a row does not see: their scores are replaced; their V must not meet the zero probabilities if it is not
// finite, so blocks on the causal edge or the sequence's end are looked through in shared memory: rows behind the
// sequence become zeros, non-finite elements too, and the (rare) latter are added to the rows that do see them at the end.
template <int HD, bool BF16, bool NEG>
__global__ void __launch_bounds__(kThreads, 1)
    packed_attention_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                            const __grid_constant__ CUtensorMap mv, const PackedArgs a) {
  using L = PackedSmem<HD>;
  constexpr int NS = L::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* Qs = smem;
  uint8_t* ring = smem + 2 * L::kQTile;
  Item* items = reinterpret_cast<Item*>(smem + L::kBars);       // [kItems]
  uint8_t* answer = reinterpret_cast<uint8_t*>(items + kItems);  // 16 bytes
  uint64_t* bar = reinterpret_cast<uint64_t*>(answer + 16);
  uint64_t* full = bar;               // [NS]
  uint64_t* empty = full + NS;        // [NS]
  uint64_t* qfull = empty + NS;       // [2]
  uint64_t* qempty = qfull + 2;       // [2]
  uint64_t* sfull = qempty + 2;       // [2][2]: tile, buffer
  uint64_t* pready = sfull + 4;       // [2][2]
  uint64_t* odone = pready + 4;       // [2][2]
  uint64_t* ifull = odone + 4;        // [kItems]
  uint64_t* iempty = ifull + kItems;  // [kItems]
  uint64_t* taken = iempty + kItems;
  uint64_t* done = taken + 1;
  int32_t* ctl = reinterpret_cast<int32_t*>(done + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctl);
  volatile int32_t* ab = ctl + 1;
  volatile int32_t* bad = ctl + 2;    // a non-finite value was taken out of an edge block of some item
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);  // tiles
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&qfull[t], 1);
      mbar_init(&qempty[t], 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sfull[2 * t + i], 1);
        mbar_init(&pready[2 * t + i], 4);  // warps
        mbar_init(&odone[2 * t + i], 1);
      }
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&ifull[i], 1);
      mbar_init(&iempty[i], 11);  // the copying thread, the issuing and the softmax warps
    }
    mbar_init(taken, 1);
    mbar_init(done, 2);
    *ab = 0;
    *bad = 0;
    *reinterpret_cast<uint64_t*>(ctl + 4) = a.wait_ns;
    mbar_fence_init();
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

  if (warp >= 8) {
    if (warp == 10) {
      int index = blockIdx.x, published = 0, asked = 0, told = 0;
      bool more = true;  // index and those behind it may be items
      while (true) {
        // (the next CTA is asked for before this item is found)
        if (index >= 0) {
          if (lane == 0) {
            mbar_arrive_expect_tx(taken, 16);
            take_over_cta(answer, taken);
          }
          ++asked;
        }
        const int s = published % kItems;
        if (published >= kItems && !mbar_wait_warp(&iempty[s], (published / kItems - 1) & 1, ab)) {
          *ab = 1;
          break;
        }
        if (index < 0) {
          if (lane == 0) {
            items[s].stop = 1;
            mbar_arrive(&ifull[s]);
          }
          break;
        }
        // (the grid is an upper bound: behind the first index without an item there is none, and the rest is only taken
        // over so that it is not launched)
        more = more && find_item(a, index, lane, &items[s]);
        if (more) {
          if (lane == 0) mbar_arrive(&ifull[s]);
          ++published;
        }
        if (!mbar_wait_warp(taken, told & 1, ab)) {
          *ab = 1;
          break;
        }
        ++told;
        index = taken_over_cta(answer);
        __syncwarp();
        fence_async_smem();  // the answer has been read before the next one is written
      }
      if (told < asked) mbar_wait(taken, told & 1, &never, a.wait_ns);  // no answer may arrive behind the CTA's end
    } else if (warp == 8) {
      if (lane == 0) {
        const uint32_t qbytes = (uint32_t)(a.tok * a.group) * 128 * (HD / 64);
        int g = 0, nq[2] = {0, 0};  // blocks and Q tiles asked for so far
        bool ok = true;
        auto block = [&](const Item& w, int j) {
          const int s = g % NS;
          if (g >= NS && !mbar_wait(&empty[s], (g / NS - 1) & 1, ab, a.wait_ns)) return false;
          mbar_arrive_expect_tx(&full[s], L::kPair);
          for (int c = 0; c < 2 * (HD / 64); ++c)
            tma_load_3d(ring + s * L::kPair + c * L::kBlock, c < HD / 64 ? &mk : &mv, c % (HD / 64) * 64, w.h, w.k0 + j * kKeys, &full[s]);
          ++g;
          return true;
        };
        for (int it = 0; ok; ++it) {
          const int s = it % kItems;
          if (!(ok = mbar_wait(&ifull[s], (it / kItems) & 1, ab, a.wait_ns))) break;
          const Item w = items[s];
          mbar_arrive(&iempty[s]);
          if (w.stop) break;
          const int n0 = item_blocks(w, 0, a.tok), n1 = item_blocks(w, 1, a.tok), n = max(n0, n1);
          for (int j = 0; ok && j < n; ++j) {
            ok = block(w, j);
            if (j > 0) continue;
            for (int t = 0; ok && t < 2; ++t) {
              if ((t ? n1 : n0) == 0) continue;
              if (nq[t] > 0 && !(ok = mbar_wait(&qempty[t], (nq[t] - 1) & 1, ab, a.wait_ns))) break;
              mbar_arrive_expect_tx(&qfull[t], qbytes);
              for (int c = 0; c < HD / 64; ++c)
                tma_load_3d(Qs + t * L::kQTile + c * L::kQBlock, &mq, c * 64, w.h * a.group, w.q0 + w.t0 + t * a.tok, &qfull[t]);
              ++nq[t];
            }
          }
        }
        if (!ok) *ab = 1;
        // no copy may still be writing this CTA's shared memory when it exits
        for (int t = 0; t < 2; ++t)
          if (nq[t] > 0) mbar_wait(&qfull[t], (nq[t] - 1) & 1, &never, a.wait_ns);
        for (int i = g > NS ? g - NS : 0; i < g; ++i) mbar_wait(&full[i % NS], (i / NS) & 1, &never, a.wait_ns);
      }
      __syncwarp();
    } else {
      // Warps 9 and 11 issue the MMAs of tile A and of tile B.  Each runs in step and an elected lane issues: the operands
      // then live in uniform registers, where a branch for one thread would move each of them there again for every MMA
      // (120 cycles an MMA, measured).  Such a warp spends about 10 cycles an instruction, so it is spared all it can be:
      // a warp for each tile, slots and phases that are carried along, and one wait for a block of K and of V.  The
      // softmax warps free the ring's slots.  Every batch of MMAs has a commit of its own and is waited for by that one:
      // a later batch's completion was seen in front of an earlier one's of another shape.
      constexpr uint32_t id_s = tc_idesc_f16(BF16, 128, kKeys);
      constexpr uint32_t id_o = tc_idesc_f16(BF16, 128, HD) | kTcIdescBMn;
      constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);
      const uint32_t t = warp == 11;
      // descriptors differ in their low words only: the start address, and V's distance between its 64-wide blocks
      const uint32_t q_lo = ((smem_u32(Qs) + t * L::kQTile) >> 4) | (1u << 16);
      const uint32_t k_lo = (smem_u32(ring) >> 4) | (1u << 16);
      const uint32_t v_lo = ((smem_u32(ring) + L::kTile) >> 4) | ((L::kBlock >> 4) << 16);
      const uint32_t tS = tmem + t * 128, tO = tmem + 256 + t * 128;
      struct Slot {
        uint32_t s, phase;
        __device__ __forceinline__ void next(uint32_t n) {
          if (++s == n) s = 0, phase ^= 1;
        }
      };
      Slot kb{0, 0};      // the ring slot of the next block to score
      uint32_t vs = 0;    // and of the next one to weigh
      uint32_t s_buf = 0, s_phase = 0, p_buf = 0, p_phase = 0, q_phase = 0;
      // S of the next block into the next buffer, once the product that read P there is done
      auto score = [&](bool last) {
        if (!mbar_wait_warp(&odone[2 * t + s_buf], s_phase ^ 1, ab)) return false;
        const uint32_t b = k_lo + kb.s * (L::kPair >> 4), d = tS + s_buf * 64;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < HD / 16; ++c)
            tc_mma_f16_lo(d, q_lo + (((c / 4) * L::kQBlock + (c % 4) * 32) >> 4), b + (((c / 4) * L::kBlock + (c % 4) * 32) >> 4), kHi,
                          id_s, c > 0);
          tc_commit(&sfull[2 * t + s_buf]);
          if (last) tc_commit(&qempty[t]);
        }
        __syncwarp();
        s_phase ^= s_buf;
        s_buf ^= 1;
        kb.next(NS);
        return true;
      };
      bool ok = true, early = false;  // early: the item's first scores have been issued in front of the last one's end
      Slot iw{0, 0};                  // the item (kItems of them)
#pragma unroll 1
      while (ok) {
        if (!(ok = mbar_wait_warp(&ifull[iw.s], iw.phase, ab))) break;
        const int stop = items[iw.s].stop;
        const int nk = stop ? 0 : item_blocks(items[iw.s], t, a.tok), other = stop ? 0 : item_blocks(items[iw.s], 1 - t, a.tok);
        __syncwarp();
        if (elect_one()) mbar_arrive(&iempty[iw.s]);
        __syncwarp();
        if (stop) break;
        iw.next(kItems);
        if (nk > 0 && !early) {
          if (!(ok = mbar_wait_warp(&qfull[t], q_phase, ab) && mbar_wait_warp(&full[kb.s], kb.phase, ab))) break;
          if (!(ok = score(nk == 1))) break;
        }
        early = false;
        q_phase ^= nk > 0;
#pragma unroll 1
        for (int j = 0; j < nk; ++j) {
          const bool last = j + 1 == nk;
          if (!last) {
            if (!(ok = mbar_wait_warp(&full[kb.s], kb.phase, ab))) break;
            if (!(ok = score(j + 2 == nk))) break;
          } else {
            // the next item's first scores if everything for them is there (and no block comes in front that only the
            // other tile sees)
            if (nk >= other && __all_sync(0xFFFFFFFFu, mbar_try_wait(&ifull[iw.s], iw.phase)) && !items[iw.s].stop) {
              const int next = item_blocks(items[iw.s], t, a.tok);
              if (next > 0 && __all_sync(0xFFFFFFFFu, mbar_try_wait(&full[kb.s], kb.phase) && mbar_try_wait(&qfull[t], q_phase))) {
                if (!(ok = score(next == 1))) break;
                early = true;
              }
            }
          }
          if (!(ok = mbar_wait_warp(&pready[2 * t + p_buf], p_phase, ab))) break;
          tc_fence_after();
          const uint32_t b = v_lo + vs * (L::kPair >> 4), p = tS + p_buf * 64;
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < kKeys / 16; ++c) tc_mma_f16_ts(tO, p + c * 8, b + c * (2048 >> 4), kHi, id_o, j > 0 || c > 0);
            tc_commit(&odone[2 * t + p_buf]);
          }
          __syncwarp();
          p_phase ^= p_buf;
          p_buf ^= 1;
          if (++vs == NS) vs = 0;
        }
        // blocks that only the other tile sees: each is waited for all the same, a barrier's phases tell only two apart
        for (int k = nk; ok && k < other; ++k) {
          ok = mbar_wait_warp(&full[kb.s], kb.phase, ab);
          kb.next(NS);
          if (++vs == NS) vs = 0;
        }
      }
      if (!ok) *ab = 1;
      if (elect_one()) tc_commit(done);  // on every path: arrives once no MMA of this warp is in flight
      __syncwarp();
    }
  } else {
    const int t = warp >> 2, r = threadIdx.x & 127;
    const int row_tok = r / a.group, row_head = r % a.group;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + t * 128, tO = tmem + lanes + 256 + t * 128;
    bool ok = true;
    uint32_t ns = 0;          // blocks of this tile so far
    uint32_t g = 0;           // ring blocks of the items before
    auto wait_all = [&](uint64_t* b, uint32_t parity) { return mbar_wait_warp(b, parity, ab); };
    for (int it = 0; ok; ++it) {
      const int is = it % kItems;
      if (!(ok = wait_all(&ifull[is], (it / kItems) & 1))) break;
      const Item w = items[is];
      if (w.stop) break;
      const int n0 = item_blocks(w, 0, a.tok), n1 = item_blocks(w, 1, a.tok);
      const int nk = t ? n1 : n0;
      const int tok = w.t0 + t * a.tok + row_tok;
      const bool live = r < a.tok * a.group && tok < w.lq;
      const int lim = min(tok + w.lk - w.lq, w.lk - 1);  // the last key that this row sees
      const int warp_lim = __reduce_min_sync(0xFFFFFFFFu, lim);
      // the first key that some row of the tiles with this block does not see: from its block on, blocks are edge blocks
      const int edge = w.t0 + w.lk - w.lq + 1 + (n0 > 0 ? 0 : a.tok);
      // the running maximum (and ms, what is subtracted from scores) and sum, and the score above which the maximum is
      // replaced (never by what stands in rows that are not the sequence's: it must not decide how the others are rounded)
      float m = -INFINITY, ms = 0.0f, l = 0.0f, limit = live ? -INFINITY : INFINITY;
      for (int j = 0; j < nk; ++j, ++ns) {
        const uint32_t buf = ns & 1;
        if (!wait_all(&sfull[2 * t + buf], (ns >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // (S(j) was issued once the product of block j - 2 was done)
        if (r == 0 && j >= 2) mbar_arrive(&empty[(g + j - 2) % NS]);
        __syncwarp();  // (the tensor-memory instructions want a warp in step)
        float x[kKeys];
        tmem_ld64(tS + buf * 64, x);
        if constexpr (NEG) {  // scale < 0
#pragma unroll
          for (int c = 0; c < kKeys; ++c) x[c] = -x[c];
        }
        const int left = lim - j * kKeys;  // columns c <= left are seen
        if (warp_lim - j * kKeys < kKeys - 1) {
#pragma unroll
          for (int c = 0; c < kKeys; ++c) x[c] = c <= left ? x[c] : -INFINITY;
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
        const bool grow = mx > limit;
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float mn = live && mx > -INFINITY ? fmaxf(m, mx * a.scale_log2) : m;
          const float f = mn == -INFINITY ? 1.0f : exp2_fast(m - mn);
          m = mn;
          ms = m == -INFINITY ? 0.0f : m - kWeightUp<BF16>;
          l *= f;
          if (live && m > -INFINITY) limit = (m + kRescale) / a.scale_log2;
          if (j > 0) {
            // block j - 1's product must be in O
            if (!wait_all(&odone[2 * t + (buf ^ 1)], ((ns - 1) >> 1) & 1)) {
              ok = false;
              break;
            }
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
        // ---- an edge block's values, looked through by both tiles (they take out the same; the block has arrived: its
        // scores are here)
        if ((j + 1) * kKeys > edge) {
          uint8_t* vt = ring + (g + j) % NS * L::kPair + L::kTile;
          const int key = r >> 1;  // two threads to a key
          auto piece = [&](int c) {
            return reinterpret_cast<uint4*>(vt + (c / 8) * L::kBlock + key * 128 + (((c & 7) ^ (key & 7)) * 16));
          };
          constexpr uint32_t kExp = BF16 ? 0x7F80u : 0x7C00u, kExp2 = kExp * 0x10001u, kOne2 = (0x8000u - kExp) * 0x10001u;
          if (j * kKeys + key >= w.lk) {
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
        const float2 sc = make_float2(a.scale_log2, a.scale_log2), nm = make_float2(-ms, -ms);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int c0 = 0; c0 < kKeys; c0 += 32) {
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 y = __ffma2_rn(make_float2(x[c0 + e], x[c0 + e + 1]), sc, nm);
            const float2 p = make_float2(exp2_fast(y.x), exp2_fast(y.y));  // (0 where x is -infinity: not seen)
            sum[(e >> 1) & 1] = __fadd2_rn(sum[(e >> 1) & 1], p);
            u[e >> 1] = pack2(p.x, p.y, BF16 ? DT_BF16 : DT_F16);
          }
          tmem_st16(tS + buf * 64 + c0 / 2, u);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[2 * t + buf]);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      // ---- O / l, behind the last two products (S(nk - 1) was issued behind the others)
      if (ok && nk > 1) ok = wait_all(&odone[2 * t + (ns & 1)], ((ns - 2) >> 1) & 1);
      if (ok && nk > 0) ok = wait_all(&odone[2 * t + (~ns & 1)], ((ns - 1) >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const int n = max(n0, n1);
      if (r == 0)  // the last two blocks, and (each once it is there) those that only the other tile sees
        for (int j = max(0, nk - 2); j < n; ++j) {
          if (j >= nk && !mbar_wait(&full[(g + j) % NS], ((g + j) / NS) & 1, ab, a.wait_ns)) *ab = 1;
          mbar_arrive(&empty[(g + j) % NS]);
        }
      g += n;
      __syncwarp();
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      uint8_t* po = a.out + (int64_t)(w.q0 + tok) * a.out_stride + (int64_t)(w.h * a.group + row_head) * HD * 2;
#pragma unroll 1
      for (int c0 = 0; c0 < HD; c0 += 32) {
        float o[32];
        if (nk > 0) {
          tmem_ld32(tO + c0, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.0f;
        }
        if (live) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = l == 0.0f ? 0.0f : o[e] * inv;
          if (*bad) {
            for (int key = max(0, edge / kKeys * kKeys); key <= lim; ++key) {
              const uint8_t* pv = a.v + (int64_t)(w.k0 + key) * a.v_stride + (int64_t)w.h * HD * 2 + c0 * 2;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float v = kv_to_f32(reinterpret_cast<const uint16_t*>(pv)[e], BF16 ? DT_BF16 : DT_F16);
                o[e] += isfinite(v) ? 0.0f : v;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) u[k] = pack2(o[e + 2 * k], o[e + 2 * k + 1], BF16 ? DT_BF16 : DT_F16);
            *reinterpret_cast<uint4*>(po + (c0 + e) * 2) = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
        __syncwarp();
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

template <int HD, bool BF16, bool NEG>
struct PackedKey {};

template <int HD, bool BF16, bool NEG>
cudaError_t packed_launch(const CUtensorMap (&m)[3], const PackedArgs& a, int64_t grid, cudaStream_t st) {
  auto* kernel = packed_attention_kernel<HD, BF16, NEG>;
  const cudaError_t e = allow_smem<PackedKey<HD, BF16, NEG>>((const void*)kernel, PackedSmem<HD>::kBytes);
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
      !encode(&m[1], n_k ? k : q, bf16, head_dim, n_kv_heads, n_k ? n_k : 1, n_k ? k_stride : kw, 1, kKeys) ||
      !encode(&m[2], n_k ? v : q, bf16, head_dim, n_kv_heads, n_k ? n_k : 1, n_k ? v_stride : kw, 1, kKeys))
    return ADP_ERR_INVALID_ARG;
  PackedArgs a{cu_q, cu_k, static_cast<const uint8_t*>(v), static_cast<uint8_t*>(out), v_stride * 2, out_stride * 2,
               n_seqs, n_q, n_k, n_kv_heads, group, tok,
               // (a scale of 0 becomes the least normal number: the scores' differences vanish all the same, and what is
               // not seen stays at -infinity)
               fmaxf(log2_scale(fabsf(scale)), kScaleMin), dev_status, packed_wait_ns(n_k, n_seqs)};
  const int64_t pairs = (int64_t)n_q / (2 * tok) + n_seqs;  // at most: every sequence may end inside a pair
  const int64_t grid = pairs * n_kv_heads;
  if (grid > 0x7FFFFFFF) return ADP_ERR_UNSUPPORTED_CONFIG;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e;
  auto by_sign = [&](auto hd, auto b) {
    constexpr int H = decltype(hd)::value;
    constexpr bool B = decltype(b)::value;
    e = scale < 0.0f ? packed_launch<H, B, true>(m, a, grid, st) : packed_launch<H, B, false>(m, a, grid, st);
  };
  auto by_type = [&](auto hd) {
    if (bf16) by_sign(hd, std::true_type());
    else by_sign(hd, std::false_type());
  };
  if (head_dim == 128) by_type(std::integral_constant<int, 128>());
  else by_type(std::integral_constant<int, 64>());
  return cuda_status(e, "adp_packed_attention");
}
