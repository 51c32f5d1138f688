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
    const bf16x2 lo = {(__bf16)v[0], (__bf16)v[1]}, hi = {(__bf16)v[2], (__bf16)v[3]};   // nearest even
    const uint2 b = make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
    if (a.vec && col + 4 <= a.N) {
      *reinterpret_cast<uint2*>(o) = b;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (col + k < a.N) o[k] = (uint16_t)((k < 2 ? b.x : b.y) >> (16 * (k & 1)));
    }
  }
}

// Eight consecutive columns: 16 bytes of bf16 in one store.
__device__ __forceinline__ void store8(const GroupedArgs& a, uint8_t* row, int col, const f32x4& u, const f32x4& v) {
  if (!a.out_f32 && a.vec && col + 8 <= a.N) {
    const bf16x8 b = {(__bf16)u[0], (__bf16)u[1], (__bf16)u[2], (__bf16)u[3],
                      (__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    *reinterpret_cast<bf16x8*>(reinterpret_cast<uint16_t*>(row) + col) = b;
  } else {
    store4(a, row, col, u);
    store4(a, row, col + 4, v);
  }
}

}  // namespace situ
