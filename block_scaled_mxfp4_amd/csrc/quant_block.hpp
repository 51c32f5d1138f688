// The E4M3 rule with one fp32 scale per 128 columns, shared by the quantization
// (quant_block.hip) and the kept activations (activation.hip).
#pragma once

#include "common.hpp"

namespace situ {

// x / s as far as its E4M3 code goes: q = x r with r = rcp(s) within an ulp, and one
// correction by the remainder x - q s.  The quotient of bf16 values and block
// maxima lies 2^-13 from every midpoint between two codes unless it is one, and at
// the midpoints the corrected value rounds as the exactly divided one (all 1449
// pairs of mantissas and distances, r an ulp off to either side, in rational
// arithmetic).  A block with an infinity has scale inf and codes of NaN; a NaN
// element gives NaN and leaves the block's scale to the others.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}

// max(amax, 2^-100) / 448, rounded as a division is (every bf16 mantissa, in rational arithmetic).
__device__ __forceinline__ float block_scale(float amax) {
  constexpr float kR = 1.0f / 448.0f;
  amax = fmaxf(amax, 0x1p-100f);
  const float q = amax * kR, s = fmaf(fmaf(-q, 448.0f, amax), kR, q);
  return amax < __builtin_inff() ? s : amax;
}

// Codes of eight elements of a block with scale s.
__device__ __forceinline__ uint2 block_codes(const float f[8], float s) {
  const float r = __builtin_amdgcn_rcpf(s);
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int d = 0;
    d = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(f[4 * i], s, r), quotient(f[4 * i + 1], s, r), d, false);
    d = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(f[4 * i + 2], s, r), quotient(f[4 * i + 3], s, r), d, true);
    o[i] = (uint32_t)d;
  }
  return make_uint2(o[0], o[1]);
}

}  // namespace situ
