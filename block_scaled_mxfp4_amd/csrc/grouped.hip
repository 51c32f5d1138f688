// Products with rows grouped by expert, tiles staged in LDS
// (situ_moe_grouped_matmul and its gradients, situ_moe_matmul_fp8_block128).
//
// out[t, c] = sum_q T(t, q) C(q, c) per group, on the matrix cores:
//  - a workgroup computes BM rows (t) x BN columns (c) and walks q in steps of
//    128 bytes of an operand row (64 bf16, 128 E4M3).  C is the MFMA's first
//    operand, so a lane holds consecutive columns of one output row;
//  - an operand whose rows run along q (x, dy and w of the forward products)
//    lies in LDS as rows of 128 bytes; one whose rows run along t or c (w of
//    dx, both operands of dw) lies as 64 rows of q, and the fragments are
//    gathered by the transposing LDS read (ds_read_b64_tr_b16: in each 16
//    lanes, lane i receives element i % 4 of the 8 bytes that lanes i / 4,
//    4 + i / 4, 8 + i / 4 and 12 + i / 4 address);
//  - stages are filled by DMA (global_load_lds), each lane with a 64-bit
//    address of its own, so gathered rows and arrays beyond 4 GiB cost
//    nothing extra.  Lanes past an edge repeat an address inside it: rows and
//    columns past the end are not stored, and elements past the end of q are
//    cleared in the fragments of the last step, in both operands;
//  - E4M3: the 16x16x128 MFMA of one step is one scale block, so its result
//    is multiplied into the accumulators by a_scale * w_scale in fp32.  (The
//    scaled MFMA takes powers of two only.)  That instruction adds the eight
//    products of each aligned 8 bytes in fixed point, dropping what lies 13
//    bits below the largest one's leading bit (measured on gfx950 by the
//    smallest addend that survives beside 2^14 at each of the 128 positions;
//    the eights' sums are then added in fp32): 1.4e-5 of a normal sum, a
//    hundredth of the bf16 rounding that follows.  Outputs in fp32 take the
//    codes as bf16, which hold them exactly, through the bf16 MFMA, whose
//    sums are fp32: half the rate.
//
// Rounding: products and sums in fp32 but for that, one rounding to bf16 at
// the store.
#include "common.hpp"
#include "dma.hpp"
#include "grouped_dev.hpp"

namespace situ {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

template <int BM_, int BN_, int WM_, int WN_, int ST_, int MINB_>
struct Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_, MINB = MINB_;
  static constexpr int W = WM * WN, TT = BM / WM / 16, CT = BN / WN / 16;
  static_assert(BM % (8 * W) == 0 && BN % (8 * W) == 0, "whole DMA blocks per wave");
  static_assert(CT % 2 == 0 && TT >= 1, "column tiles go in pairs");
};

constexpr int kMaxE = 1024;

__device__ __forceinline__ void gdma16(const uint8_t* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               ::"s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p) : "memory", "m0");
}
__device__ __forceinline__ void gdma4(const void* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               ::"s"(__builtin_amdgcn_readfirstlane(lds)), "v"(p) : "memory", "m0");
}

struct Tile {
  int e, m0, n0;      // group, first row / column of the tile (kGWgrad: m0 a row of dw)
  int lo, hi;         // rows of the group (kGWgrad: of the contraction)
};

// Swizzles: the 16-byte slot of a chunk within a 128-byte row.  Rows read
// together by eight lanes get eight slots.
__device__ __forceinline__ int swz_t(int row) { return row & 7; }
__device__ __forceinline__ int swz_c(int row) { return (row & 3) | ((row >> 1) & 4); }

// The elements 8 d .. 8 d + 7 of q that lie below `valid`, as masks of bf16 pairs.
__device__ __forceinline__ uint32_t pair_mask(int valid, int d) {
  return valid >= 2 * d + 2 ? 0xffffffffu : (valid == 2 * d + 1 ? 0xffffu : 0u);
}

template <class C, int MODE>
struct Kernel {
  static constexpr bool kX = MODE == kGFwd8x, kF8 = MODE == kGFwd8 || kX, kWg = MODE == kGWgrad;
  static constexpr bool kTRows = !kWg;                          // T rows run along q
  static constexpr bool kCRows = MODE == kGFwd || kF8;
  static constexpr int kTBytes = C::BM * 128, kCBytes = C::BN * 128;
  static constexpr int kSBytes = kF8 ? (C::BM + 63) / 64 * 256 + 256 : 0;   // scales of a step
  static constexpr int kStage = kTBytes + kCBytes + kSBytes;
  static constexpr int kTD = C::BM / 8 / C::W, kCD = C::BN / 8 / C::W;   // DMAs of a wave and step
  static constexpr int kThreads = C::W * 64;
  static constexpr int kIds = kWg ? 8 * 64 * 4 : 0;             // ring of row indices, 64 per step
  static_assert(!kF8 || (C::BM + 63) / 64 < C::W, "a wave for each 64 row scales and one for the block scales");

  // Byte offset, within an operand stored as 64 rows of q and R columns, of
  // the 16-byte slot holding the chunk of columns 8 c .. + 7 of row r: units
  // of 16 columns are permuted so that the eight rows half a wave reads
  // together lie in different banks.
  template <int R>
  static __device__ __forceinline__ int unit_slot(int r, int u) {
    return u ^ (((r & 3) | ((r >> 1) & 4)) & (R / 16 - 1));
  }

  struct Geo {
    const uint8_t* t[kTD];     // kTRows: row address + chunk; else operand + column chunk
    const uint8_t* c[kCD];
    const float* s;            // kF8: this lane's scale at step 0
    int t_chunk, c_chunk;      // byte of the lane's chunk within a step
  };

  static __device__ __forceinline__ Geo geometry(const GroupedArgs& a, const Tile& x, int wave, int lane) {
    Geo g{};
    if constexpr (kTRows) {
      g.t_chunk = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
      for (int i = 0; i < kTD; ++i) {
        const int r = min(x.m0 + (wave + C::W * i) * 8 + (lane >> 3), x.hi - 1);
        const int row = max(index_row(a.t_div, a.pairs, r, a.t_rows), 0);
        g.t[i] = a.t + (int64_t)row * a.t_stride + g.t_chunk;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kTD; ++i) {
        const int p = (wave + C::W * i) * 64 + lane, r = p / (C::BM / 8), s = p % (C::BM / 8);
        const int col = x.m0 + 16 * unit_slot<C::BM>(r, s >> 1) + 8 * (s & 1);
        g.t[i] = a.t + 2 * (col < a.M ? col : 0);
      }
    }
    const uint8_t* w = a.c + (int64_t)(kWg ? 0 : x.e) * a.c_expert;
    if constexpr (kCRows) {
      g.c_chunk = ((lane & 7) ^ swz_c(8 * wave + (lane >> 3))) * 16;   // W is even: the same for every i
#pragma unroll
      for (int i = 0; i < kCD; ++i) {
        const int n = min(x.n0 + (wave + C::W * i) * 8 + (lane >> 3), a.N - 1);
        g.c[i] = w + (int64_t)n * a.c_stride + g.c_chunk;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kCD; ++i) {
        const int p = (wave + C::W * i) * 64 + lane, r = p / (C::BN / 8), s = p % (C::BN / 8);
        const int col = x.n0 + 16 * unit_slot<C::BN>(r, s >> 1) + 8 * (s & 1);
        g.c[i] = w + 2 * (col < a.N ? col : 0);
      }
    }
    if constexpr (kF8) {
      constexpr int kTW = (C::BM + 63) / 64;
      if (wave < kTW) {
        const int r = min(x.m0 + 64 * wave + lane, x.hi - 1);
        const int row = max(index_row(a.t_div, a.pairs, r, a.t_rows), 0);
        g.s = a.t_scale + (int64_t)row * a.ts_stride;
      } else {                       // one per 128 columns of the tile, lane after lane
        const int nb = (a.N + 127) / 128, kb = (a.K + 127) / 128;
        g.s = a.c_scale + ((int64_t)x.e * nb + min(x.n0 / 128 + lane, nb - 1)) * kb;
      }
    }
    return g;
  }

  // Request step j into the stage at `st`.
  template <bool IDX>
  static __device__ __forceinline__ void issue(const GroupedArgs& a, const Tile& x, const Geo& g, uint32_t st,
                                               const uint8_t* ids, int j, int wave, int lane) {
    if constexpr (IDX) {             // the row indices of a later step go ahead of this step's rows
      const int s = j + C::ST - 1;
      gdma4(a.pairs + min(x.lo + 64 * (int64_t)s + lane, (int64_t)x.hi - 1), lds_addr_of(ids) + (s & 7) * 256);
    }
    const int64_t q = (int64_t)j * 128;
    if constexpr (kTRows) {
      // a chunk past the end of q repeats the row's first one
      const int64_t at = q + g.t_chunk < (int64_t)a.K * (kF8 ? 1 : 2) ? q : -g.t_chunk;
#pragma unroll
      for (int i = 0; i < kTD; ++i) gdma16(g.t[i] + at, st + (wave + C::W * i) * 1024);
    } else {
#pragma unroll
      for (int i = 0; i < kTD; ++i) {
        const int r = ((wave + C::W * i) * 64 + lane) / (C::BM / 8);
        gdma16(g.t[i] + q_row<IDX>(a, x, a.t_div, a.t_rows, ids, j, r) * a.t_stride, st + (wave + C::W * i) * 1024);
      }
    }
    if constexpr (kCRows) {
      const int64_t at = q + g.c_chunk < (int64_t)a.K * (kF8 ? 1 : 2) ? q : -g.c_chunk;
#pragma unroll
      for (int i = 0; i < kCD; ++i) gdma16(g.c[i] + at, st + kTBytes + (wave + C::W * i) * 1024);
    } else {
#pragma unroll
      for (int i = 0; i < kCD; ++i) {
        const int r = ((wave + C::W * i) * 64 + lane) / (C::BN / 8);
        const int64_t row = kWg ? q_row<IDX>(a, x, a.c_div, a.c_rows, ids, j, r) : min(64 * j + r, a.K - 1);
        gdma16(g.c[i] + row * a.c_stride, st + kTBytes + (wave + C::W * i) * 1024);
      }
    }
    if constexpr (kF8) {
      constexpr int kTW = (C::BM + 63) / 64;
      gdma4(g.s + j, st + kTBytes + kCBytes + min(wave, kTW) * 256);
    }
  }
  static constexpr int dmas(bool idx) { return kTD + kCD + (kF8 ? 1 : 0) + (idx ? 1 : 0); }

  // kGWgrad: the matrix row of element r of step j.
  template <bool IDX>
  static __device__ __forceinline__ int64_t q_row(const GroupedArgs& a, const Tile& x, const RowDiv& d, int n_rows,
                                                  const uint8_t* ids, int j, int r) {
    if constexpr (IDX) {
      if (d.div != 0) {
        const int p = max(reinterpret_cast<const int32_t*>(ids)[(j & 7) * 64 + r], 0);
        return min(row_of(d, p), n_rows - 1);
      }
    }
    return min((int64_t)x.lo + 64 * (int64_t)j + r, (int64_t)x.hi - 1);
  }

  // Eight consecutive elements of q (half h of a step, group g of lanes) of
  // the 16 columns of unit u, from an operand stored as 64 rows of q.
  template <int R>
  static __device__ __forceinline__ uint4 read_tr(const uint8_t* base, int u, int h, int lane) {
    const int l = lane & 15, g = lane >> 4;
    uint4 v;
    uint32_t* d = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int r = 32 * h + 8 * g + 4 * p + (l >> 2);
      const uint8_t* at = base + r * (2 * R) + unit_slot<R>(r, u) * 32 + (l & 3) * 8;
      const s16x4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4*)(uintptr_t)lds_addr_of(at));
      const uint2 w2 = __builtin_bit_cast(uint2, w);
      d[2 * p] = w2.x;
      d[2 * p + 1] = w2.y;
    }
    return v;
  }

  // Multiply one staged step into the accumulators; TAIL: `left` elements of
  // q remain in it, the others are cleared.
  template <bool TAIL>
  static __device__ __forceinline__ void compute(const uint8_t* st, int wm, int wn, int lane, int left,
                                                 f32x4 (&acc)[C::CT][C::TT]) {
    const int l = lane & 15, g = lane >> 4;
    const int t0 = wm * C::TT, c0 = wn * C::CT;     // the wave's first 16-row and 16-column tiles
    auto clear = [&](uint4& v, int h) {
      if constexpr (TAIL) {
        uint32_t* d = reinterpret_cast<uint32_t*>(&v);
        const int valid = kF8 ? left - 16 * (4 * h + g) : left - 32 * h - 8 * g;
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] &= kF8 ? (valid > 0 ? 0xffffffffu : 0u) : pair_mask(valid, i);
      }
    };
    auto read_t = [&](int j, int h) {
      uint4 v;
      if constexpr (kTRows) {
        v = *reinterpret_cast<const uint4*>(st + (16 * (t0 + j) + l) * 128 + (((g + 4 * h) ^ swz_t(l)) * 16));
      } else {
        v = read_tr<C::BM>(st, t0 + j, h, lane);
      }
      clear(v, h);
      return v;
    };
    auto read_c = [&](int i, int h) {
      uint4 v;
      if constexpr (kCRows) {
        // tiles 2 p and 2 p + 1 share 32 columns: row 4 a + b of them is column 8 a + b and 8 a + 4 + b, so a
        // lane's results are eight consecutive columns
        const int row = 16 * (c0 + (i & ~1)) + 8 * (l >> 2) + (l & 3) + 4 * (i & 1);
        v = *reinterpret_cast<const uint4*>(st + kTBytes + row * 128 + (((g + 4 * h) ^ swz_c(row)) * 16));
      } else {
        v = read_tr<C::BN>(st + kTBytes, c0 + i, h, lane);
      }
      clear(v, h);
      return v;
    };
    if constexpr (kF8) {
      const float* sc = reinterpret_cast<const float*>(st + kTBytes + kCBytes);
      float ts[C::TT];
      uint4 cv[C::CT][2];
      float cs[C::CT];
#pragma unroll
      for (int i = 0; i < C::CT; ++i) {
        cv[i][0] = read_c(i, 0);
        cv[i][1] = read_c(i, 1);
        cs[i] = sc[(C::BM + 63) / 64 * 64 + (c0 + i) / 8];
      }
#pragma unroll
      for (int j = 0; j < C::TT; ++j) ts[j] = sc[16 * (t0 + j) + l];
#pragma unroll
      for (int j = 0; j < C::TT; ++j) {
        const uint4 lo = read_t(j, 0), hi = read_t(j, 1);
        const i32x8 tv = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
#pragma unroll
        for (int i = 0; i < C::CT; ++i) {
          const i32x8 v = {(int)cv[i][0].x, (int)cv[i][0].y, (int)cv[i][0].z, (int)cv[i][0].w,
                           (int)cv[i][1].x, (int)cv[i][1].y, (int)cv[i][1].z, (int)cv[i][1].w};
          f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
          if constexpr (kX) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8x8_to_bf16x8(v[2 * q], v[2 * q + 1]),
                                                          fp8x8_to_bf16x8(tv[2 * q], tv[2 * q + 1]), p, 0, 0, 0);
          } else {
            p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, tv, p, 0, 0, 0, 0, 0, 0);
          }
          const float s = ts[j] * cs[i];
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][j][k] = fmaf(p[k], s, acc[i][j][k]);
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bf16x8 cv[C::CT];
#pragma unroll
        for (int i = 0; i < C::CT; ++i) cv[i] = __builtin_bit_cast(bf16x8, read_c(i, h));
#pragma unroll
        for (int j = 0; j < C::TT; ++j) {
          const bf16x8 tv = __builtin_bit_cast(bf16x8, read_t(j, h));
#pragma unroll
          for (int i = 0; i < C::CT; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cv[i], tv, acc[i][j], 0, 0, 0);
        }
      }
    }
  }

  static __device__ __forceinline__ void epilogue(const GroupedArgs& a, const Tile& x, int wm, int wn, int lane,
                                                  f32x4 (&acc)[C::CT][C::TT]) {
    const int l = lane & 15, g = lane >> 4;
#pragma unroll
    for (int j = 0; j < C::TT; ++j) {
      const int t = x.m0 + 16 * (wm * C::TT + j) + l;
      if (t >= (kWg ? a.M : x.hi)) continue;
      const int row = kWg ? t : index_row(a.o_div, a.pairs, t, a.o_rows);
      if (row < 0) continue;
      uint8_t* o = static_cast<uint8_t*>(a.out) + (kWg ? (int64_t)x.e * a.out_expert : 0) + (int64_t)row * a.out_stride;
      const int n0 = x.n0 + 16 * wn * C::CT;
#pragma unroll
      for (int i = 0; i < C::CT; ++i) {
        const int col = n0 + (kCRows ? 16 * (i & ~1) + 8 * g + 4 * (i & 1) : 16 * i + 4 * g);
        store4(a, o, col, acc[i][j]);
      }
    }
  }
};

// Exclusive prefix of the groups' row tiles in pre[0 .. E].
template <int NT>
__device__ __forceinline__ void tile_prefix(const GroupedArgs& a, int bm, int* pre, int* part, int tid) {
  constexpr int kPer = kMaxE / NT;
  int cnt[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    int lo = 0, hi = 0;
    if (e < a.experts) group_rows(a, e, lo, hi);
    cnt[i] = (hi - lo + bm - 1) / bm;
    sum += cnt[i];
  }
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int up = __shfl_up(inc, d, kWave);
    if ((tid & 63) >= d) inc += up;
  }
  if ((tid & 63) == 63) part[tid >> 6] = inc;
  __syncthreads();
  int at = inc - sum;
  for (int w = 0; w < (tid >> 6); ++w) at += part[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e <= a.experts) pre[e] = at;
    at += cnt[i];
  }
  if (tid == NT - 1 && a.experts == kMaxE) pre[kMaxE] = at;
  __syncthreads();
}

// The group whose tiles hold m: the last e with pre[e] <= m (every group
// after it that starts there is empty, so pre[e] <= m < pre[e + 1]).
__device__ __forceinline__ int find_group(const int* pre, int experts, int m, int lane) {
  const int c = pre[min(16 * lane, experts)];
  const int chunk = __popcll(__ballot(16 * lane < experts && c <= m)) - 1;
  const int e = 16 * chunk + (lane & 15);
  const int v = pre[min(e, experts)];
  return 16 * chunk + (__popcll(__ballot(e < experts && v <= m)) >> 2) - 1;
}

template <class C, int MODE, bool IDX>
__global__ __launch_bounds__(C::W * 64, C::MINB) void grouped_kernel(GroupedArgs a) {
  using K = Kernel<C, MODE>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::ST * K::kStage + K::kIds + (kMaxE + 1 + 16) * 4];
  uint8_t* ids = lds + C::ST * K::kStage;
  int* pre = reinterpret_cast<int*>(lds + C::ST * K::kStage + K::kIds);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const uint32_t lds0 = lds_addr_of(lds);

  int m_tiles;
  if constexpr (K::kWg) {
    m_tiles = a.experts * a.m_bound;
  } else {
    if (a.offsets) {
      tile_prefix<K::kThreads>(a, C::BM, pre, pre + kMaxE + 1, tid);
      m_tiles = min(pre[a.experts], a.m_bound);   // ascending offsets never exceed the bound
    } else {
      m_tiles = a.m_bound;
    }
  }
  const int64_t total = (int64_t)m_tiles * a.n_tiles;

  // each XCD (workgroups b, b + 8, ...) walks a contiguous share of the tiles
  const int xcds = min((int)gridDim.x, 8), xcd = blockIdx.x % xcds, slots = gridDim.x / xcds;
  const int64_t first = total * xcd / xcds, last = total * (xcd + 1) / xcds;
  for (int64_t it = first + blockIdx.x / xcds; it < last; it += slots) {
    Tile x;
    int steps, left;
    if constexpr (K::kWg) {
      const int per = a.m_bound * a.n_tiles;
      x.e = (int)(it / per);
      const int r = (int)(it % per);
      x.m0 = (r % a.m_bound) * C::BM;
      x.n0 = (r / a.m_bound) * C::BN;
      group_rows(a, x.e, x.lo, x.hi);
      steps = (x.hi - x.lo + 63) / 64;
      left = x.hi - x.lo - 64 * (steps - 1);
    } else {
      // within a group: eight row tiles by all column tiles, rows fastest
      int local, m_l;
      if (a.offsets) {
        x.e = find_group(pre, a.experts, (int)(it / a.n_tiles), lane);
        x.e = __builtin_amdgcn_readfirstlane(x.e);
        local = (int)(it - (int64_t)pre[x.e] * a.n_tiles);
        m_l = pre[x.e + 1] - pre[x.e];
      } else {
        x.e = 0;
        local = (int)it;
        m_l = m_tiles;
      }
      group_rows(a, x.e, x.lo, x.hi);
      const int block = local / (8 * a.n_tiles), in = local % (8 * a.n_tiles);
      const int high = min(8, m_l - 8 * block);
      x.m0 = x.lo + (8 * block + in % high) * C::BM;
      x.n0 = (in / high) * C::BN;
      if (x.m0 >= x.hi || x.n0 >= a.N) continue;   // only with offsets that do not ascend
      constexpr int kQ = K::kF8 ? 128 : 64;
      steps = (a.K + kQ - 1) / kQ;
      left = a.K - kQ * (steps - 1);
    }
    const bool tail = left < (K::kF8 ? 128 : 64);

    f32x4 acc[C::CT][C::TT];
#pragma unroll
    for (int i = 0; i < C::CT; ++i)
#pragma unroll
      for (int j = 0; j < C::TT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    if (steps > 0) {
      const typename K::Geo g = K::geometry(a, x, wave, lane);
      __syncthreads();                             // the last tile's stages have been read
      if constexpr (IDX) {
        for (int s = wave; s < C::ST - 1; s += C::W)
          reinterpret_cast<int32_t*>(ids)[s * 64 + lane] = a.pairs[min(x.lo + 64 * s + lane, x.hi - 1)];
        __syncthreads();
      }
#pragma unroll
      for (int s = 0; s < C::ST - 1; ++s)
        if (s < steps) K::template issue<IDX>(a, x, g, lds0 + s * K::kStage, ids, s, wave, lane);
      int stage = 0;
      for (int j = 0; j < steps; ++j) {
        constexpr int kD = K::dmas(IDX);
        const int after = min(C::ST - 2, steps - 1 - j);
        if (after >= 2) dma_barrier<2 * kD>();
        else if (after == 1) dma_barrier<kD>();
        else dma_barrier<0>();
        const int ahead = stage == 0 ? C::ST - 1 : stage - 1;
        if (j + C::ST - 1 < steps)
          K::template issue<IDX>(a, x, g, lds0 + ahead * K::kStage, ids, j + C::ST - 1, wave, lane);
        const uint8_t* st = lds + stage * K::kStage;
        if (tail && j == steps - 1) K::template compute<true>(st, wm, wn, lane, left, acc);
        else K::template compute<false>(st, wm, wn, lane, left, acc);
        stage = stage + 1 == C::ST ? 0 : stage + 1;
      }
    }
    K::epilogue(a, x, wm, wn, lane, acc);
  }
}

template <class C, int MODE, bool IDX>
hipError_t launch_as(GroupedArgs& a, int cus, hipStream_t s) {
  a.n_tiles = (a.N + C::BN - 1) / C::BN;
  int64_t tiles;
  if (MODE == kGWgrad) {
    a.m_bound = (a.M + C::BM - 1) / C::BM;
    tiles = (int64_t)a.m_bound * a.n_tiles * a.experts;
  } else {
    a.m_bound = a.offsets ? a.rows / C::BM + a.experts : (a.rows + C::BM - 1) / C::BM;
    tiles = (int64_t)a.m_bound * a.n_tiles;
  }
  const int64_t most = (int64_t)C::MINB * 4 / C::W * cus;    // resident workgroups
  int64_t grid = tiles < most ? tiles : most;
  if (grid > 8) grid = (grid + 7) / 8 * 8;
  hipLaunchKernelGGL((grouped_kernel<C, MODE, IDX>), dim3((unsigned)grid), dim3(C::W * 64), 0, s, a);
  return hipGetLastError();
}

using Mid = Cfg<64, 128, 2, 2, 3, 2>;

}  // namespace

hipError_t launch_grouped(GroupedMode mode, GroupedArgs& a, int cus, hipStream_t s) {
  if (mode == kGFwd8 && a.out_f32) mode = kGFwd8x;
  if ((mode == kGFwd || mode == kGFwd8 || mode == kGFwd8x) && few_rows(a)) return launch_grouped_few(mode, a, cus, s);
  switch (mode) {
    case kGFwd: return launch_as<Mid, kGFwd, false>(a, cus, s);
    case kGFwd8: return launch_as<Mid, kGFwd8, false>(a, cus, s);
    case kGFwd8x: return launch_as<Mid, kGFwd8x, false>(a, cus, s);
    case kGDgrad: return launch_as<Mid, kGDgrad, false>(a, cus, s);
    case kGWgrad:
      if (a.pairs && (a.t_div.div || a.c_div.div)) return launch_as<Mid, kGWgrad, true>(a, cus, s);
      return launch_as<Mid, kGWgrad, false>(a, cus, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace situ
