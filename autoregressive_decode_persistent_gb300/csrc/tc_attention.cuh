// What the kernels of attention on the tensor cores have in common: waits of whole warps, offsets of packed rows, tensor maps.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "device.cuh"
#include "paged.cuh"
#include "tc.cuh"

namespace adp {
namespace {

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
__device__ __forceinline__ bool mbar_wait_warp_loop(uint64_t* b, uint32_t parity, volatile int32_t* abort) {
  uint64_t t0 = 0;  // (the clock is asked late: reading it takes longer than most waits)
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(b, parity))) return true;
    if ((it & 63) == 0) {
      const uint64_t now = globaltimer();
      if (t0 == 0) t0 = now;
      if (__any_sync(0xFFFFFFFFu, *abort != 0 || now - t0 > wait_limit(abort))) return false;
    }
  }
}
__device__ __noinline__ bool mbar_wait_warp_slow(uint64_t* b, uint32_t parity, volatile int32_t* abort) {
  return mbar_wait_warp_loop(b, parity, abort);
}
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* b, uint32_t parity, volatile int32_t* abort) {
  return __all_sync(0xFFFFFFFFu, mbar_try_wait(b, parity)) ? true : mbar_wait_warp_slow(b, parity, abort);
}
// The same without a call, for kernels that share out their registers (whose calls would need the largest share), and as short
// as can be: the kernel's loops have to stay in the instruction cache.  Its limit, in 2^20 cycles, lies 8 bytes behind the abort word.
__device__ __forceinline__ bool mbar_wait_warp_inline(uint64_t* b, uint32_t parity, volatile int32_t* abort) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(b, parity))) return true;
  const uint32_t t0 = (uint32_t)(clock64() >> 20);
  do {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(b, parity))) return true;
  } while (__all_sync(0xFFFFFFFFu, *abort == 0 && (uint32_t)(clock64() >> 20) - t0 <= (uint32_t)abort[2]));
  return false;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// fp16 weights are held 2^7 times larger (and so is their sum): up to 2^15 beside a maximum that is stale by 2^8, they stay
// below fp16's 65,504, and a weight keeps all its bits down to 2^-21 of the largest and some down to 2^-32, where 2^-14 and
// 2^-25 would let the tail of a long context vanish beside one dominating key.  (bf16 has fp32's range.)
template <bool BF16>
constexpr float kWeightUp = BF16 ? 0.0f : 7.0f;

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
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
inline bool encode(CUtensorMap* map, const void* base, bool bf16, int hd, int heads, int64_t rows, int64_t stride, int box_heads,
            int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)hd, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)hd * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, one[3] = {1, 1, 1};
  return encode_fn()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                     const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace adp
