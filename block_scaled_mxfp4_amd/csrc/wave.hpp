// Reductions over the 64 lanes of a wave, by DPP moves in the registers (no
// LDS round trip as a shuffle takes): steps of 1, 2, 4, 8 within rows of 16
// lanes, then a row's last lane to the next row, then lane 31 to the upper half;
// lane 63 holds the result (others hold sums of no use).  Every lane must be
// active.  The order is fixed.
#pragma once

#include "common.hpp"

namespace situ {

// LDS that other lanes of the wave read or wrote: in order, once the compiler keeps it so.
__device__ __forceinline__ void wave_lds() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The wave of a workgroup, as a value the compiler knows to be the same in all lanes.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave)); }

template <int kCtrl>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111>(v);
  v = dpp_add<0x112>(v);
  v = dpp_add<0x114>(v);
  v = dpp_add<0x118>(v);
  v = dpp_add<0x142>(v);
  v = dpp_add<0x143>(v);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, true);   // 0 from outside
  return v > o ? v : o;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0x111>(v);
  v = dpp_max<0x112>(v);
  v = dpp_max<0x114>(v);
  v = dpp_max<0x118>(v);
  v = dpp_max<0x142>(v);
  v = dpp_max<0x143>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The sum of lane l and lane l ^ 32, in both.
__device__ __forceinline__ uint32_t halves_sum(uint32_t v) {
  const auto both = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return both[0] + both[1];
}

}  // namespace situ
