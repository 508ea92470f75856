// The block-scaled FP8 format of rbq_fp8_quant.cu, rbq_fp8_gemm.cu and
// rbq_fp8_wgrad.cu: E4M3 codes with one power-of-two scale per block.
//
//   value = code * s,  s = 2^(b - 127),  b one byte (E8M0, as OCP MX names it)
//   s = the smallest power of two with amax / s <= 448 (the largest E4M3
//       value), and at least 2^-117; amax = the block's largest finite |x|.
//
// Why powers of two and not amax / 448 itself: the tensor cores multiply E8M0
// scales in (tcgen05 kind::mxf8f6f4), so a scaled product costs what a plain
// one does; x / s is exact, so a code carries one rounding and not two; and
// code * s is exact in BF16 (4 significant bits), which is what the gradient
// kernels feed their MMAs.  E4M3 is a floating-point format: up to the
// binade of its subnormals the larger step between scales costs no accuracy.
// The floor 2^-117 keeps every decoded value (down to 2^-9 s) a normal BF16
// number; a block of zeros gets it.  At the other end, |x| of 248 * 2^120
// (3.296e38) and more rounds to the code of 2^128, which BF16 and fp32 hold as
// infinity.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rbq_sm100.cuh"

namespace rbq {
namespace fp8 {

constexpr int kBlock = 128;            // values per scale along a row (and rows per scale of a weight)
constexpr int kMaxSize = 1 << 30;      // rows and columns of an operand: block counts and coordinates stay in 32 bits
constexpr uint32_t kMinScale = 10;     // 2^-117
constexpr uint32_t kMaxScale = 247;    // 2^120: amax up to the largest fp32

__host__ __device__ constexpr int blocks(int n) { return (n + kBlock - 1) / kBlock; }

// E8M0 byte of a block whose largest finite magnitude is amax (>= 0): with
// amax = m 2^(p - 127), 448 = 1.75 2^8, the exponent is p - 127 - 8, one more
// when m > 1.75.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int b = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(min(max(b, static_cast<int>(kMinScale)), static_cast<int>(kMaxScale)));
}
// 2^(127 - b), the factor from values to codes, and 2^(b - 127), for b in
// [kMinScale, kMaxScale] both normal numbers.
__device__ __forceinline__ float inv_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }
// 2^(b - 127) for any byte: 0 is 2^-127 (a subnormal), 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t b) {
  if (b == 0u) return __uint_as_float(0x00400000u);
  return b == 255u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(b << 23);
}

// Four values -> four E4M3 bytes (round to nearest even; NaN -> 0x7F).
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
// Two E4M3 bytes -> two values.
__device__ __forceinline__ float2 decode2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xFFFFu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Two fp32 (their bits) -> one word of two BF16.
__device__ __forceinline__ uint32_t bf16x2(uint32_t lo, uint32_t hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// True in one thread of a converged warp, the one that issues its MMAs or its
// TMA copies.  Issued under a test of the lane number a tcgen05.mma took 173
// cycles whatever its size; a 256 x 256 x 32 one runs for 128, and takes those
// under elect.sync.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0u;
}
// Arrive on an mbarrier of any CTA of the cluster, ordering nothing but the
// execution: for a warp that has read tensor memory (tcgen05.wait::ld and
// tcgen05.fence::before_thread_sync order those reads) and hands its columns back.
// A releasing arrival would also wait for the warp's stores to global memory.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
// A box of a tensor map from shared to global memory (what lies outside the
// tensor is left out), as a bulk group of its own.
__device__ __forceinline__ void tma_store_2d(const void* tmap, int x, int y, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(static_cast<uint32_t>(__cvta_generic_to_shared(src)))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_3d(const void* tmap, int x, int y, int z, const void* src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z), "r"(static_cast<uint32_t>(__cvta_generic_to_shared(src)))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the last N of this thread's bulk groups have read their shared
// memory; all of them have been written.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// As mbar_warp_wait, for a barrier that threads of the other CTA arrive on.
__device__ __forceinline__ bool mbar_warp_wait_cl(uint64_t* bar, uint32_t parity, volatile uint32_t* abort) {
  return !__any_sync(0xffffffffu, !sm100::mbar_wait_or_abort_cl(bar, parity, abort));
}
// The warp's number, in a form that the compiler knows to be the same in all its threads.
__device__ __forceinline__ int warp_number() { return __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0); }

}  // namespace fp8
}  // namespace rbq
