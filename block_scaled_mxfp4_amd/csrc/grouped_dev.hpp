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

// Four consecutive columns of an output row; one rounding for bf16.  Stores of 16
// bytes pass the caches by (16 groups of 1024 rows, dw 1536 x 3584 in fp32: 234 us
// and 212; adapter rows 768 wide: 15.6 and 13.9).
__device__ __forceinline__ void store4(const GroupedArgs& a, uint8_t* row, int col, const f32x4& v) {
  if (a.out_f32) {
    float* o = reinterpret_cast<float*>(row) + col;
    if (a.vec && col + 4 <= a.N) {
      __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(o));
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

// Eight consecutive columns of a bf16 row, already rounded.
__device__ __forceinline__ void store8(const GroupedArgs& a, uint8_t* row, int col, const uint4& b) {
  uint16_t* o = reinterpret_cast<uint16_t*>(row) + col;
  if (a.vec && col + 8 <= a.N) {
    __builtin_nontemporal_store(__builtin_bit_cast(i32x4, b), reinterpret_cast<i32x4*>(o));
  } else {
    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (col + k < a.N) o[k] = (uint16_t)(w[k / 2] >> (16 * (k % 2)));
  }
}
__device__ __forceinline__ uint4 pack8(const f32x4& u, const f32x4& v) {
  const bf16x8 b = {(__bf16)u[0], (__bf16)u[1], (__bf16)u[2], (__bf16)u[3],
                    (__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};   // nearest even
  return __builtin_bit_cast(uint4, b);
}

// The other lane's value of each pair of lanes 2 i, 2 i + 1 (every lane active).
__device__ __forceinline__ uint32_t swap_pair(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
}
__device__ __forceinline__ uint4 swap_pair(const uint4& v) {
  return make_uint4(swap_pair(v.x), swap_pair(v.y), swap_pair(v.z), swap_pair(v.w));
}
__device__ __forceinline__ uint4 pick(bool c, const uint4& u, const uint4& v) {
  return make_uint4(c ? u.x : v.x, c ? u.y : v.y, c ? u.z : v.z, c ? u.w : v.w);
}

}  // namespace situ
