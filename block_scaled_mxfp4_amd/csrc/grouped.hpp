// Interfaces of the products with rows grouped by expert (grouped.hip): the
// bf16 product, its two gradients and the E4M3 product with scales per 128.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace situ {

// floor(n / div) for 0 <= n < 2^31 as (n * mul) >> (31 + s) with s =
// ceil(log2 div), mul = floor(2^(31 + s) / div) + 1: mul * div exceeds
// 2^(31 + s) by at most div <= 2^s, so the error n * 2^s / 2^(31 + s) stays
// below 1 / div.  div = 1 divides by nothing; div = 0 marks an operand whose
// rows are in group order (no index).
struct RowDiv {
  uint32_t div, mul, shift;
};
inline RowDiv make_row_div(int32_t d) {
  RowDiv r{(uint32_t)d, 0, 0};
  if (d < 2) return r;
  uint32_t s = 0;
  while ((1ull << s) < (uint64_t)d) ++s;
  r.mul = (uint32_t)(((1ull << (31 + s)) / (uint64_t)d) + 1);
  r.shift = s - 1;
  return r;
}

enum GroupedMode : int { kGFwd = 0, kGFwd8 = 1, kGDgrad = 2, kGWgrad = 3, kGFwd8x = 4 };

// out[t, c] = sum_q T(t, q) C(q, c), per group.  Strides in bytes.
//   kGFwd    T = x rows (q = k), C = w[e] rows n           out [rows, n]
//   kGFwd8   the same on E4M3 codes with scales per 128 along k
//   kGFwd8x  kGFwd8 with the products of a block summed in fp32 (fp32 outputs)
//   kGDgrad  T = dy rows (q = n), C = w[e] columns k       out [rows, k]
//   kGWgrad  T = dy columns n, C = x columns k, q = the group's rows; out [E, n, k]
struct GroupedArgs {
  const uint8_t* t;
  int64_t t_stride;
  const uint8_t* c;
  int64_t c_stride, c_expert;
  const float* t_scale;       // kGFwd8: [rows, ceil(K / 128)]
  int64_t ts_stride;          // floats
  const float* c_scale;       // kGFwd8: [E, ceil(N / 128), ceil(K / 128)]
  const int32_t* offsets;     // [E + 1], or null: one group of all rows
  const int32_t* pairs;       // [rows] or null
  RowDiv t_div, c_div, o_div; // row of T / C / out for position r: r (div 0) or pairs[r] / div
  int32_t t_rows, c_rows, o_rows;
  int32_t rows, experts;
  int32_t M;                  // kGWgrad: n
  int32_t N, K;               // output columns; contraction length (kGWgrad: unused)
  void* out;
  int64_t out_stride, out_expert;   // bytes
  int32_t out_f32;
  int32_t vec;                // rows of out start on 16 bytes
  int32_t m_bound;            // tiles of rows there can be at most (kGWgrad: tiles of n)
  int32_t n_tiles;
};

hipError_t launch_grouped(GroupedMode mode, GroupedArgs& a, int cus, hipStream_t s);
// The kernel (and tile) launch_grouped takes.
const char* grouped_kernel_name(GroupedMode mode, const GroupedArgs& a, int cus);

// The forward products where groups hold few rows (grouped_few.hip).
bool few_rows(const GroupedArgs& a);
bool few_wide(const GroupedArgs& a, int cus);
hipError_t launch_grouped_few(GroupedMode mode, GroupedArgs& a, int cus, hipStream_t s);

struct QuantBlockArgs {
  const uint16_t* x;
  int64_t x_stride;           // elements
  uint8_t* codes;
  float* scales;
  int64_t rows;
  int32_t cols;
};
hipError_t launch_quant_block128(const QuantBlockArgs& a, hipStream_t s);

}  // namespace situ
