// The forward products grouped by expert where groups hold few rows: the
// weights are read once and their stream is the time.
//
// out[r, n] = sum_k x[r, k] w[e, n, k] (and the E4M3 form, grouped.hip).  A
// workgroup owns 8 CB columns of one expert and all of the expert's rows, up
// to 32 at a time, so the expert comes from the block index and no list of
// tiles is built.  Its waves split k between them, step by step (128 bytes of
// a row), each holding its fragments in registers straight from memory with
// U steps in flight; the partial sums are added in LDS in the waves' order.
//
// A load takes 8 weight rows x 128 bytes, whole cache lines: loads of 16 rows
// x 64 bytes, the matrix core's own order, streamed 4.0 TB/s where these reach
// 5.0 (112 groups of 2.3 rows, 768 x 3584 E4M3: 80 us and 54).  The 16 x 32 operand (four 8-element chunks of 16 rows)
// is then filled with both halves of 8 rows: row r < 8 holds chunks 0 .. 3 of
// weight row r and row 8 + r chunks 4 .. 7, and only products with the same
// half of x count:
//  - up to 8 rows of x: column t holds chunks 0 .. 3 of x row t, column 8 + t
//    chunks 4 .. 7; the diagonal quarters of the result are wanted;
//  - more: one product with each half of 16 rows of x, the upper or the lower
//    half of each result being wanted.
// The matrix cores have the time to compute what is not wanted.
//
// E4M3 codes are taken as bf16, which hold them exactly, so that the sums are
// fp32 for every output type; a block of 128 is one step.
#include <algorithm>

#include "grouped_dev.hpp"

namespace situ {

namespace {

template <bool F8, int NWK, int CB>
struct Few {
  static constexpr int kLds = NWK * CB * 64;      // f32x4 of one pass's partial sums

  static __device__ __forceinline__ void keep(uint4& v, uint32_t m) {
    v.x &= m;
    v.y &= m;
    v.z &= m;
    v.w &= m;
  }
  // acc += C T over one chunk of each lane (8 bf16 or 16 E4M3 elements)
  static __device__ __forceinline__ f32x4 mfma(const uint4& c, const uint4& t, f32x4 acc) {
    if constexpr (F8) {
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8x8_to_bf16x8(c.x, c.y), fp8x8_to_bf16x8(t.x, t.y), acc, 0, 0, 0);
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8x8_to_bf16x8(c.z, c.w), fp8x8_to_bf16x8(t.z, t.w), acc, 0, 0, 0);
    } else {
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, c), __builtin_bit_cast(bf16x8, t), acc,
                                                     0, 0, 0);
    }
  }

  // Rows [m0, min(m0 + 16 MT, hi)), or up to 8 rows (MT 0), times the columns.
  template <int MT, int U>
  static __device__ __forceinline__ void pass(const GroupedArgs& a, int e, int m0, int hi, int n0, int wk, int lane,
                                              f32x4* part) {
    constexpr int NT = MT ? MT : 1, NH = MT ? 2 : 1;          // row tiles, halves of x held apart
    constexpr int NA = !F8 && MT ? 2 : 1;                     // accumulators per tile
    const int l = lane & 15, g = lane >> 4;
    const int kb = a.K * (F8 ? 1 : 2), steps = (kb + 127) / 128;
    const int c_chunk = 64 * (l >> 3) + 16 * g;               // byte of this lane's weight chunk in a step
    const uint8_t* tp[NT];
    const float* tsp[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = min(m0 + 16 * j + (MT ? l : l & 7), hi - 1);
      const int row = max(index_row(a.t_div, a.pairs, r, a.t_rows), 0);
      tp[j] = a.t + (int64_t)row * a.t_stride;
      if constexpr (F8) tsp[j] = a.t_scale + (int64_t)row * a.ts_stride;
    }
    const uint8_t* cp[CB];
#pragma unroll
    for (int i = 0; i < CB; ++i)
      cp[i] = a.c + (int64_t)e * a.c_expert + (int64_t)min(n0 + 8 * i + (l & 7), a.N - 1) * a.c_stride;
    const float* csp = nullptr;
    if constexpr (F8) csp = a.c_scale + ((int64_t)e * ((a.N + 127) / 128) + n0 / 128) * steps;
    f32x4 acc[CB][NT][NA];
#pragma unroll
    for (int i = 0; i < CB; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < NA; ++h) acc[i][j][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // U steps s0, s0 + NWK, ...; `edge`: some lie past the end of k, or the
    // row's last chunks do: those chunks repeat the row's first one and are
    // cleared, in both operands and the scales
    auto run = [&](int s0, bool edge) {
      uint4 c[U][CB], t[U][NT][NH];
      float ts[U][NT], cs[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int s = s0 + u * NWK;
        const int at = 128 * s + c_chunk;
#pragma unroll
        for (int i = 0; i < CB; ++i)
          c[u][i] = *reinterpret_cast<const uint4*>(cp[i] + (!edge || at < kb ? at : 0));
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const int th = MT ? 128 * s + 64 * h + 16 * g : at;
#pragma unroll
          for (int j = 0; j < NT; ++j)
            t[u][j][h] = *reinterpret_cast<const uint4*>(tp[j] + (!edge || th < kb ? th : 0));
        }
        if constexpr (F8) {
          const int sc = edge ? min(s, steps - 1) : s;
          cs[u] = csp[sc];
#pragma unroll
          for (int j = 0; j < NT; ++j) ts[u][j] = tsp[j][sc];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (edge) {
          const int s = s0 + u * NWK;
          const uint32_t m = 128 * s + c_chunk < kb ? 0xffffffffu : 0u;
#pragma unroll
          for (int i = 0; i < CB; ++i) keep(c[u][i], m);
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const uint32_t mh = MT ? (128 * s + 64 * h + 16 * g < kb ? 0xffffffffu : 0u) : m;
#pragma unroll
            for (int j = 0; j < NT; ++j) keep(t[u][j][h], mh);
          }
          if constexpr (F8) {
            cs[u] = s < steps ? cs[u] : 0.0f;
#pragma unroll
            for (int j = 0; j < NT; ++j) ts[u][j] = s < steps ? ts[u][j] : 0.0f;
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < CB; ++i) {
            if constexpr (F8) {
              const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
              f32x4 p = mfma(c[u][i], t[u][j][0], z);
              if constexpr (NH == 2) {
                const f32x4 q = mfma(c[u][i], t[u][j][1], z);
#pragma unroll
                for (int k = 0; k < 4; ++k) p[k] = g < 2 ? p[k] : q[k];
              }
              const float f = ts[u][j] * cs[u];
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[i][j][0][k] = fmaf(p[k], f, acc[i][j][0][k]);
            } else {
#pragma unroll
              for (int h = 0; h < NH; ++h) acc[i][j][h] = mfma(c[u][i], t[u][j][h], acc[i][j][h]);
            }
          }
      }
    };
    int s = wk;
    for (; 128 * (s + (U - 1) * NWK) + 128 <= kb; s += U * NWK) run(s, false);
    if (s < steps) run(s, true);

    // add the waves' partial sums and the two halves of k: lanes g < 2 of a
    // tile hold the lower half of columns 4 g .. + 3, lanes g + 2 the upper
    // (and with up to 8 rows, x row t the lower and column 8 + t the upper)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        f32x4 v = acc[i][j][0];
        if constexpr (NA == 2) {
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = g < 2 ? v[k] : acc[i][j][1][k];
        }
        part[(wk * CB + i) * 64 + lane] = v;
      }
      __syncthreads();
      for (int q = wk * 64 + lane; q < CB * 32; q += NWK * 64) {    // 4 columns of one row each
        const int i = q / 32, gg = (q >> 4) & 1, r = q & 15;
        if (!MT && r >= 8) continue;
        const int t = m0 + 16 * j + r;
        if (t >= hi) continue;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < NWK; ++w)
          v += part[(w * CB + i) * 64 + 16 * gg + r] + part[(w * CB + i) * 64 + 16 * (gg + 2) + (MT ? r : r + 8)];
        const int row = index_row(a.o_div, a.pairs, t, a.o_rows);
        if (row >= 0)
          store4(a, static_cast<uint8_t*>(a.out) + (int64_t)row * a.out_stride, n0 + 8 * i + 4 * gg, v);
      }
      __syncthreads();
    }
  }
};

template <bool F8, int NWK, int CB>
__global__ __launch_bounds__(NWK * 64) void grouped_few_kernel(GroupedArgs a) {
  using F = Few<F8, NWK, CB>;
  __shared__ f32x4 part[F::kLds];
  const int lane = threadIdx.x & 63, wk = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = blockIdx.x / a.n_tiles, n0 = (blockIdx.x % a.n_tiles) * 8 * CB;
  int lo, hi;
  group_rows(a, e, lo, hi);
  for (int m0 = lo; m0 < hi; m0 += 32) {
    const int left = hi - m0;
    if (left <= 8) F::template pass<0, 4>(a, e, m0, hi, n0, wk, lane, part);
    else if (left <= 16) F::template pass<1, 2>(a, e, m0, hi, n0, wk, lane, part);
    else F::template pass<2, 2>(a, e, m0, hi, n0, wk, lane, part);
  }
}

template <bool F8, int NWK, int CB>
hipError_t launch_as(GroupedArgs& a, hipStream_t s) {
  a.n_tiles = (a.N + 8 * CB - 1) / (8 * CB);
  hipLaunchKernelGGL((grouped_few_kernel<F8, NWK, CB>), dim3((unsigned)a.n_tiles * (unsigned)a.experts),
                     dim3(NWK * 64), 0, s, a);
  return hipGetLastError();
}

template <bool F8>
hipError_t launch_type(GroupedArgs& a, int cus, hipStream_t s) {
  return few_wide(a, cus) ? launch_as<F8, 4, 4>(a, s) : launch_as<F8, 8, 2>(a, s);
}

}  // namespace

// Up to four rows a group on average, or eight in all.  From there on groups of
// more than eight rows take the 16-row passes, whose x costs as much as w, and
// the tiles of grouped.hip are as fast or faster (8 groups, 4096 x 4096 bf16:
// 8 rows each 80 us here, 62 there; 32 groups, 1536 x 2048 E4M3: 27 and 23).
// One workgroup for each group and 16 columns has to fit a grid.
bool few_rows(const GroupedArgs& a) {
  return a.rows <= std::max<int64_t>(8, 4 * (int64_t)a.experts) && (int64_t)a.experts * ((a.N + 15) / 16) <= 1 << 22;
}

// Sixteen columns a workgroup of eight waves where the columns of 32 would
// leave CUs idle, else 32 columns and four waves.
bool few_wide(const GroupedArgs& a, int cus) {
  return (int64_t)a.experts * ((a.N + 31) / 32) >= 2 * (int64_t)cus;
}

hipError_t launch_grouped_few(GroupedMode mode, GroupedArgs& a, int cus, hipStream_t s) {
  return mode == kGFwd ? launch_type<false>(a, cus, s) : launch_type<true>(a, cus, s);
}

}  // namespace situ
