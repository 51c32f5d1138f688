// The weighted sum of each token's expert rows and its gradients
// (situ_moe_combine, situ_moe_combine_backward).
//
// Both move rows and compute little: HBM bounds them (8192 tokens of an EP8 shard,
// 16 x 3584: 29 us, 6.1 TB/s, part of it from the caches; the gradients of 4095 x 16
// x 3584: 185 us, 5.2 TB/s).  A lane takes eight columns
// (16 bytes of bf16), a wave 512 at once.  The token's rows and weights are read by its
// first lanes together, those that are not local drop out of a ballot, and the
// others' rows are requested four at a time from addresses the whole wave shares.
// Local weights of 0 are products too, as the formula has them.
#include <algorithm>

#include "routed.hpp"
#include "wave.hpp"

namespace situ {

namespace {

constexpr int kCols = 512;            // of a wave at once
// Of them a wave of the sum takes two (8192 tokens, an eighth of 16 x 3584: 29.2 us; one 31.2, four 31.2).
constexpr int kPieces = 2;
constexpr int kAtOnce = 4;            // rows requested together
constexpr int kWaves = 4;             // of a workgroup

template <bool F32>
struct Eight { uint4 a; };
template <>
struct Eight<true> { uint4 a, b; };

template <bool F32>
__device__ __forceinline__ Eight<F32> load8(const void* p, int64_t at) {
  if constexpr (F32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
    return {q[0], q[1]};
  } else {
    return {*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at)};
  }
}
// The gradient's y is read once (4095 x 16 x 3584: 195 us with ordinary loads, 185 so).
template <bool F32>
__device__ __forceinline__ Eight<F32> load8_once(const void* p, int64_t at) {
  const i32x4* q = reinterpret_cast<const i32x4*>(static_cast<const char*>(p) + at * (F32 ? 4 : 2));
  if constexpr (F32)
    return {__builtin_bit_cast(uint4, __builtin_nontemporal_load(q)),
            __builtin_bit_cast(uint4, __builtin_nontemporal_load(q + 1))};
  else
    return {__builtin_bit_cast(uint4, __builtin_nontemporal_load(q))};
}
template <bool F32>
__device__ __forceinline__ void widen(const Eight<F32>& v, float f[8]) {
  const uint32_t w[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
  if constexpr (F32) {
    const uint32_t u[4] = {v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) { f[i] = __uint_as_float(w[i]); f[4 + i] = __uint_as_float(u[i]); }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_to_f32(w[i] & 0xffffu);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t at, const float f[8]) {
  if constexpr (F32) {
    float* q = static_cast<float*>(p) + at;
    *reinterpret_cast<f32x4*>(q) = f32x4{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<f32x4*>(q + 4) = f32x4{f[4], f[5], f[6], f[7]};
  } else {
    const bf16x8 b = {(__bf16)f[0], (__bf16)f[1], (__bf16)f[2], (__bf16)f[3],
                      (__bf16)f[4], (__bf16)f[5], (__bf16)f[6], (__bf16)f[7]};   // nearest even
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = __builtin_bit_cast(uint4, b);
  }
}

// Lane i's slot first + i of a token (those before `end`): its row, -1 if it is not local, and weight.
__device__ __forceinline__ void load_slot(const situ_moe_combine_t& p, int64_t t, int slot, int end, int& row, float& w) {
  row = -1;
  w = 0.0f;
  if (slot < end) {
    const int64_t at = t * p.top_k + slot;
    row = p.inv[at];
    if (row >= p.rows) row = -1;
    w = p.weights_dtype == SITU_OUT_F32 ? static_cast<const float*>(p.weights)[at]
                                        : bf16_to_f32(static_cast<const uint16_t*>(p.weights)[at]);
  }
}
__device__ __forceinline__ int next_bit(uint64_t& m) {
  const int i = __ffsll((unsigned long long)m) - 1;
  m &= m - 1;
  return i;
}

template <bool YF, bool OF>
__global__ __launch_bounds__(64 * kWaves) void pair_combine_kernel(situ_moe_combine_t p, int parts, int64_t items) {
  const int lane = lane_id();
  for (int64_t item = (int64_t)blockIdx.x * kWaves + wave_id(); item < items; item += (int64_t)gridDim.x * kWaves) {
    const int64_t t = (uint32_t)item / (uint32_t)parts;         // items: kPieces times 512 columns of a token
    const int col = (int)(item - t * parts) * kCols * kPieces + 8 * lane;
    float acc[kPieces][8] = {};
    for (int first = 0; first < p.top_k; first += kWave) {
      int row;
      float w;
      load_slot(p, t, first + lane, p.top_k, row, w);
      uint64_t local = __ballot(row >= 0);
      while (local) {
        Eight<YF> v[kAtOnce][kPieces];
        float wt[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          wt[i] = 0.0f;
#pragma unroll
          for (int o = 0; o < kPieces; ++o) v[i][o] = Eight<YF>{};
          if (local) {
            const int s = next_bit(local);
            wt[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), s));
            const int64_t r = __builtin_amdgcn_readlane(row, s);
#pragma unroll
            for (int o = 0; o < kPieces; ++o)
              if (col + kCols * o < p.hidden) v[i][o] = load8<YF>(p.y, r * p.y_stride + col + kCols * o);
          }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
          for (int o = 0; o < kPieces; ++o) {
            float f[8];
            widen<YF>(v[i][o], f);
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[o][c] = fmaf(wt[i], f[c], acc[o][c]);
          }
      }
    }
#pragma unroll
    for (int o = 0; o < kPieces; ++o)
      if (col + kCols * o < p.hidden) store8<OF>(p.out, t * p.out_stride + col + kCols * o, acc[o]);
  }
}

// A wave takes `slots` slots of a token and walks the columns for four of its
// local ones at a time: d_out is read once for the four.
template <bool YF, bool OF>
__global__ __launch_bounds__(64 * kWaves) void pair_combine_backward_kernel(situ_moe_combine_t p, int slots, int parts,
                                                                            int64_t items) {
  const int lane = lane_id();
  for (int64_t item = (int64_t)blockIdx.x * kWaves + wave_id(); item < items; item += (int64_t)gridDim.x * kWaves) {
    const int64_t t = (uint32_t)item / (uint32_t)parts;
    const int first = (int)(item - t * parts) * slots, end = min(first + slots, p.top_k);
    int row;
    float w, mine = 0.0f;                            // lane i: the gradient of slot first + i
    load_slot(p, t, first + lane, end, row, w);
    uint64_t local = __ballot(row >= 0);
    while (local) {
      int64_t r[kAtOnce];
      float wt[kAtOnce], dot[kAtOnce];
      int slot[kAtOnce], n = 0;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        dot[i] = 0.0f;
        if (local) {
          slot[i] = next_bit(local);
          n = i + 1;
        } else {
          slot[i] = slot[0];
        }
        wt[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), slot[i]));
        r[i] = __builtin_amdgcn_readlane(row, slot[i]);
      }
      for (int col = 8 * lane; col < p.hidden; col += kCols) {
        float d[8];
        const Eight<OF> vd = load8<OF>(p.out, t * p.out_stride + col);
        Eight<YF> v[kAtOnce];
        if (p.d_weights) {
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i)
            if (i < n) v[i] = load8_once<YF>(p.y, r[i] * p.y_stride + col);
        }
        widen<OF>(vd, d);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          if (i < n) {
            if (p.d_weights) {
              float f[8];
              widen<YF>(v[i], f);
#pragma unroll
              for (int c = 0; c < 8; ++c) dot[i] = fmaf(d[c], f[c], dot[i]);
            }
            if (p.dy) {
              float f[8];
#pragma unroll
              for (int c = 0; c < 8; ++c) f[c] = wt[i] * d[c];
              store8<YF>(p.dy, r[i] * p.dy_stride + col, f);
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (i < n) {
          const float s = wave_sum(dot[i]);
          if (lane == slot[i]) mine = s;
        }
      }
    }
    if (p.d_weights && first + lane < end) p.d_weights[t * p.top_k + first + lane] = mine;
  }
}

unsigned grid_of(int64_t items) { return (unsigned)std::min<int64_t>((items + kWaves - 1) / kWaves, 1 << 16); }

}  // namespace

hipError_t launch_pair_combine(const situ_moe_combine_t& p, hipStream_t s) {
  const int parts = (p.hidden + kPieces * kCols - 1) / (kPieces * kCols);
  const int64_t items = (int64_t)p.tokens * parts;
  const dim3 grid(grid_of(items)), threads(64 * kWaves);
  const bool yf = p.y_dtype == SITU_OUT_F32, of = p.out_dtype == SITU_OUT_F32;
  if (yf && of) hipLaunchKernelGGL((pair_combine_kernel<true, true>), grid, threads, 0, s, p, parts, items);
  else if (yf) hipLaunchKernelGGL((pair_combine_kernel<true, false>), grid, threads, 0, s, p, parts, items);
  else if (of) hipLaunchKernelGGL((pair_combine_kernel<false, true>), grid, threads, 0, s, p, parts, items);
  else hipLaunchKernelGGL((pair_combine_kernel<false, false>), grid, threads, 0, s, p, parts, items);
  return hipGetLastError();
}

hipError_t launch_pair_combine_backward(const situ_moe_combine_t& p, hipStream_t s) {
  // few tokens: four slots a wave, all CUs; many: whole tokens
  int slots = std::min(p.top_k, kWave);
  while (slots > kAtOnce && (int64_t)p.tokens * ((p.top_k + slots - 1) / slots) < 8192) slots = (slots + 1) / 2;
  const int parts = (p.top_k + slots - 1) / slots;
  const int64_t items = (int64_t)p.tokens * parts;
  const dim3 grid(grid_of(items)), threads(64 * kWaves);
  const bool yf = p.y_dtype == SITU_OUT_F32, of = p.out_dtype == SITU_OUT_F32;
  if (yf && of) hipLaunchKernelGGL((pair_combine_backward_kernel<true, true>), grid, threads, 0, s, p, slots, parts, items);
  else if (yf) hipLaunchKernelGGL((pair_combine_backward_kernel<true, false>), grid, threads, 0, s, p, slots, parts, items);
  else if (of) hipLaunchKernelGGL((pair_combine_backward_kernel<false, true>), grid, threads, 0, s, p, slots, parts, items);
  else hipLaunchKernelGGL((pair_combine_backward_kernel<false, false>), grid, threads, 0, s, p, slots, parts, items);
  return hipGetLastError();
}

}  // namespace situ
