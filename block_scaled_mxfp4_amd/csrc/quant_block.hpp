// The E4M3 rule with one fp32 scale per 128 columns, shared by the quantization
// (quant_block.hip) and the kept activations (activation.hip).
#pragma once

#include "common.hpp"

namespace situ {

// x / s correctly rounded where it counts: q = x * rcp(s) is within two ulp, and
// one correction by the remainder x - q s lands on the nearest fp32.  Only in
// blocks with a maximum below 2^-98 can the remainder of an element 2^13 or more
// below it leave the normal range, and the quotient be an ulp off; its E4M3 code
// is the same (every pair of bf16 mantissas at 22 exponent distances, in
// rational arithmetic).  A block with an infinity has scale inf and codes
// of NaN; a NaN element gives NaN and leaves the block's scale to the others.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}

__device__ __forceinline__ float block_scale(float amax) { return fmaxf(amax, 0x1p-100f) / 448.0f; }

// Codes of eight elements of a block with scale s.
__device__ __forceinline__ uint2 block_codes(const float f[8], float s) {
  const float r = 1.0f / s;
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
