// E4M3 quantization of bf16 rows with one fp32 scale per row and 128 columns
// (situ_moe_quantize_fp8_block128).
//
// scale = max(amax, 2^-100) / 448; code = E4M3 round-to-nearest-even of
// x / scale.  The floor keeps an all-zero block's scale a normal number, so
// neither the quotient nor a product with the scale leaves fp32's range.
//
// The kernel moves 3 bytes per element and computes little.  Sixteen lanes
// share one block, eight elements (16 bytes) each, so a wave reads four
// blocks as 1 KB of whole lines; the block maximum takes four shuffles.
#include <algorithm>

#include "common.hpp"
#include "grouped.hpp"

namespace situ {

namespace {

// x / s correctly rounded for the values met here: q = x * rcp(s) is within
// two ulp, and one correction by the exact remainder x - q s lands on the
// nearest fp32 (s >= 2^-109 and |q| <= 448 (1 + 2^-23) keep every step in the
// normal range or exact).  A block with an infinity has scale inf and codes
// of NaN; a NaN element gives NaN and leaves the block's scale to the others.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}

__global__ __launch_bounds__(256) void quant_block128_kernel(QuantBlockArgs a, int64_t n) {
  const int nb = (a.cols + 127) / 128;
  // n is a multiple of 16: the sixteen lanes of a block leave the loop together
  for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < n; c += (int64_t)gridDim.x * 256) {   // (row, block, sixteenth)
    const int64_t rb = c >> 4;
    const int64_t row = rb / nb;
    const int b = (int)(rb - row * nb);
    const int col = b * 128 + (int)(c & 15) * 8;
    const bool in = col < a.cols;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (in) v = *reinterpret_cast<const uint4*>(a.x + row * a.x_stride + col);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_to_f32(w[i] & 0xffffu);
      f[2 * i + 1] = bf16_to_f32(w[i] >> 16);
      amax = fmaxf(amax, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
    }
#pragma unroll
    for (int m = 1; m < 16; m *= 2) amax = fmaxf(amax, __shfl_xor(amax, m, kWave));
    if (!in) continue;
    const float scale = fmaxf(amax, 0x1p-100f) / 448.0f;
    const float r = 1.0f / scale;
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int d = 0;
      d = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(f[4 * i], scale, r), quotient(f[4 * i + 1], scale, r), d, false);
      d = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(f[4 * i + 2], scale, r), quotient(f[4 * i + 3], scale, r), d, true);
      o[i] = (uint32_t)d;
    }
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    __builtin_nontemporal_store(i32x2{(int)o[0], (int)o[1]}, reinterpret_cast<i32x2*>(a.codes + row * a.cols + col));
    if ((c & 15) == 0) a.scales[rb] = scale;
  }
}

}  // namespace

hipError_t launch_quant_block128(const QuantBlockArgs& a, hipStream_t s) {
  const int64_t n = a.rows * ((a.cols + 127) / 128) * 16;
  if (n == 0) return hipSuccess;
  const int64_t blocks = std::min<int64_t>((n + 255) / 256, 1 << 20);
  hipLaunchKernelGGL(quant_block128_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, n);
  return hipGetLastError();
}

}  // namespace situ
