// Row quantisation arithmetic shared by the query quantiser, the index-K
// writer and the KV writer: the FP16 scale of a row and the 8-bit code (INT8
// or E4M3) of a value under it.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

namespace qli {
namespace {

// x / sf in FP32, rounded to nearest even, from y = RN(1 / sf): the product
// q0 = RN(x * y) is within about an ulp of the quotient, so the residual
// x - q0 * sf is exact in one FMA and RN(q0 + residual * y) is the correctly
// rounded quotient (Markstein's correction step: P. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", IBM J. Res.
// Dev. 34(1), 1990). Inputs are BF16 values and FP16 scales, so the domain
// is finite: qli_check_quant_rounding compares every pair with IEEE
// division.
__device__ __forceinline__ float quotient(float x, float sf, float y) {
  const float q0 = __fmul_rn(x, y);
  const float r = __fmaf_rn(-q0, sf, x);
  return __fmaf_rn(r, y, q0);
}

__device__ __forceinline__ int code_of(float x, float sf, float y) {
  // clamped before the conversion (same result as clamping the integer)
  return __float2int_rn(fminf(fmaxf(quotient(x, sf, y), -127.0f), 127.0f));
}

// FP16(amax / qmax) with the FP32 quotient rounded to nearest even, through
// the same correction step from RN(1/qmax) (qmax 127, or 448 for E4M3);
// capped at the largest finite FP16. The check entry point compares it with
// IEEE division for every BF16 amax.
template <bool kFp8>
__device__ __forceinline__ uint16_t scale_bits_of(float amax) {
  const float qmax = kFp8 ? 448.0f : 127.0f;
  const float rcp = kFp8 ? __uint_as_float(0x3b124925u)    // FP32 nearest 1/448
                         : __uint_as_float(0x3c010204u);   // FP32 nearest 1/127
  const float q = quotient(amax, qmax, rcp);
  uint16_t sb = __half_as_ushort(__float2half_rn(q));
  if (sb == 0x7c00u) sb = 0x7bffu;    // +inf: the largest finite FP16
  return sb;
}

// Two FP32 values to E4M3 codes (round to nearest even, saturated to the
// largest finite magnitude 448): the low byte holds lo's code.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t code_byte(float x, float sf, float y) {
  return static_cast<uint32_t>(code_of(x, sf, y)) & 0xffu;
}

}  // namespace
}  // namespace qli
