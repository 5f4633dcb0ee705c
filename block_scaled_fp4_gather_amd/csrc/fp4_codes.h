// MXFP4 codes of bf16 values, shared by the quantiser (fp4_quant.hip) and the
// linear map's own quantisation of its tokens (fp4_linear.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "decode.h"

namespace moe {

// Scale byte of a block from its largest magnitude's fp32 bits (an integer
// maximum, so that a NaN or an infinity compares above every number): 2^(
// floor(log2 amax) - 2), at least 2^-127, or 255 (NaN).
__device__ __forceinline__ uint32_t mxfp4_scale_byte(uint32_t amax_bits) {
  return amax_bits < 0x7F800000u ? (uint32_t)max((int)(amax_bits >> 23) - 2, 0) : 255u;
}

// The scale of a finite byte as the operand of the conversions, which take its
// exponent field (0: 2^-127).
__device__ __forceinline__ float mxfp4_scale(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 0x00400000u); }

// Largest magnitude's fp32 bits of 8 bf16 values.
__device__ __forceinline__ uint32_t amax8(const uint4& raw) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(max(m, (w[i] << 16) & 0x7FFFFFFFu), w[i] & 0x7FFF0000u);
  return m;
}

// E2M1 codes of 8 bf16 values over their block's scale, first value in the low
// nibble: the conversion divides by the power of two, rounds to nearest-even
// and caps magnitudes at 6 (checked for every bf16 value).
__device__ __forceinline__ uint32_t mxfp4_codes8(const uint4& raw, uint32_t byte) {
  if (byte == 255u) return 0x77777777u;
  const float s = mxfp4_scale(byte);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(raw.x), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(raw.y), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(raw.z), s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(raw.w), s, 3);
  return w;
}

}  // namespace moe
