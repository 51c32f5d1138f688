// E4M3 quantization of bf16 rows with one fp32 scale per row and 128 columns
// (situ_moe_quantize_fp8_block128).
//
// scale = max(amax, 2^-100) / 448; code = E4M3 round-to-nearest-even of
// x / scale.  The floor keeps an all-zero block's scale a normal number, so
// neither the quotient nor a product with the scale leaves fp32's range.
//
// The kernel moves 3 bytes per element and computes little.  Sixteen lanes
// share one block, eight elements (16 bytes) each, so a wave reads four
// blocks as 1 KB of whole lines; the block maximum takes four shuffles.  Four
// pieces a thread are requested together: 32768 x 3584 in 62 us (5.7 TB/s), 72
// with one.
#include <algorithm>

#include "common.hpp"
#include "grouped.hpp"

namespace situ {

namespace {

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

constexpr int kAtOnce = 4;   // pieces a thread requests before it computes

__global__ __launch_bounds__(256) void quant_block128_kernel(QuantBlockArgs a, int64_t n) {
  const int nb = (a.cols + 127) / 128;
  const int64_t all = (int64_t)gridDim.x * 256;
  // piece c: sixteenth c % 16 of block c / 16.  n is a multiple of 16: the
  // sixteen lanes of a block take every branch together
  for (int64_t c0 = (int64_t)blockIdx.x * 256 + threadIdx.x; c0 < n; c0 += kAtOnce * all) {
    uint4 v[kAtOnce];
    int64_t at[kAtOnce];
    bool in[kAtOnce];
#pragma unroll
    for (int p = 0; p < kAtOnce; ++p) {
      const int64_t c = c0 + p * all, rb = c >> 4;
      in[p] = false;
      v[p] = make_uint4(0, 0, 0, 0);
      if (c >= n) continue;
      const int64_t row = rb >> 31 ? rb / nb : (int64_t)((uint32_t)rb / (uint32_t)nb);
      const int col = (int)(rb - row * nb) * 128 + (int)(c & 15) * 8;
      in[p] = col < a.cols;
      at[p] = row * a.cols + col;
      if (in[p]) v[p] = *reinterpret_cast<const uint4*>(a.x + row * a.x_stride + col);
    }
#pragma unroll
    for (int p = 0; p < kAtOnce; ++p) {
      const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
      float f[8], amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_to_f32(w[i] & 0xffffu);
        f[2 * i + 1] = bf16_to_f32(w[i] >> 16);
        amax = fmaxf(amax, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
      }
#pragma unroll
      for (int m = 1; m < 16; m *= 2) amax = fmaxf(amax, __shfl_xor(amax, m, kWave));
      if (!in[p]) continue;
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
      __builtin_nontemporal_store(i32x2{(int)o[0], (int)o[1]}, reinterpret_cast<i32x2*>(a.codes + at[p]));
      const int64_t c = c0 + p * all;
      if ((c & 15) == 0) a.scales[c >> 4] = scale;
    }
  }
}

}  // namespace

hipError_t launch_quant_block128(const QuantBlockArgs& a, hipStream_t s) {
  const int64_t n = a.rows * ((a.cols + 127) / 128) * 16;
  if (n == 0) return hipSuccess;
  // small matrices: a piece a thread, all CUs; large ones: kAtOnce pieces a thread
  const int64_t pieces = (n + 255) / 256;
  const int64_t blocks = pieces <= 2048 ? pieces : std::min<int64_t>((pieces + kAtOnce - 1) / kAtOnce, 1 << 20);
  hipLaunchKernelGGL(quant_block128_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, n);
  return hipGetLastError();
}

}  // namespace situ
