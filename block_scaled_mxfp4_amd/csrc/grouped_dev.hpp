// Device helpers shared by the products grouped by expert (grouped.hip,
// grouped_few.hip).
#pragma once

#include "common.hpp"
#include "grouped.hpp"

namespace situ {

__device__ __forceinline__ int row_of(const RowDiv& d, int pair) {
  return d.div == 1 ? pair : (int)(__umulhi((uint32_t)pair, d.mul) >> d.shift);
}
// Row of a matrix for position r of the group order (-1: outside it).
__device__ __forceinline__ int index_row(const RowDiv& d, const int32_t* pairs, int r, int n_rows) {
  if (d.div == 0) return r;
  const int p = pairs[r];
  const int row = p < 0 ? -1 : row_of(d, p);
  return row < n_rows ? row : -1;
}

// First and one-past-last row of group e.  Offsets that do not ascend within
// [0, rows] give wrong groups, never a row outside [0, rows).
__device__ __forceinline__ void group_rows(const GroupedArgs& a, int e, int& lo, int& hi) {
  if (!a.offsets) { lo = 0; hi = a.rows; return; }
  lo = min(max(a.offsets[e], 0), a.rows);
  hi = min(max(a.offsets[e + 1], lo), a.rows);
}

// Four consecutive columns of an output row; one rounding for bf16.
__device__ __forceinline__ void store4(const GroupedArgs& a, uint8_t* row, int col, const f32x4& v) {
  if (a.out_f32) {
    float* o = reinterpret_cast<float*>(row) + col;
    if (a.vec && col + 4 <= a.N) {
      *reinterpret_cast<f32x4*>(o) = v;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (col + k < a.N) o[k] = v[k];
    }
  } else {
    uint16_t* o = reinterpret_cast<uint16_t*>(row) + col;
    uint32_t b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) b[k] = f32_to_bf16_rne(v[k]);
    if (a.vec && col + 4 <= a.N) {
      *reinterpret_cast<uint2*>(o) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (col + k < a.N) o[k] = (uint16_t)b[k];
    }
  }
}

}  // namespace situ
