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
//  - stages are filled by DMA (global_load_lds), each lane with an address of
//    its own (64 bits, or a uniform base and 32 where that reaches), so
//    gathered rows cost nothing extra.  Lanes past an edge repeat an address
//    inside it: rows and columns past the end are not stored, and elements
//    past the end of q are cleared in the fragments of the last step, in both
//    operands;
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
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.hpp"
#include "dma.hpp"
#include "grouped_dev.hpp"

namespace situ {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// PERM: a lane's results are eight consecutive columns also where C's rows run
// along q (see read_c).
template <int BM_, int BN_, int WM_, int WN_, int ST_, int MINB_, bool PERM_ = false>
struct Cfg {
  static constexpr bool PERM = PERM_;
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
template <class T>
__device__ __forceinline__ const T* uniform(const T* p) {
  const uint64_t u = (uint64_t)p;
  return reinterpret_cast<const T*>((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)u) |
                                    (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32)) << 32);
}
// The same from a uniform base and a lane's offset.
__device__ __forceinline__ void gdma16s(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               ::"s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(uniform(base)) : "memory", "m0");
}
__device__ __forceinline__ void gdma4s(const float* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               ::"s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(uniform(base)) : "memory", "m0");
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

// The elements 2 d and 2 d + 1 of q that lie below `valid`, as a mask of a bf16 pair.
__device__ __forceinline__ uint32_t pair_mask(int valid, int d) {
  return valid >= 2 * d + 2 ? 0xffffffffu : (valid == 2 * d + 1 ? 0xffffu : 0u);
}

// WIDE: rows of T (and of C in kGWgrad) may lie anywhere in their array;
// otherwise within 4 GiB of a tile's first row, or of the array's where they
// are gathered (narrow_ok), and a lane's address is a uniform base and 32 bits.
template <class C, int MODE, bool WIDE>
struct Kernel {
  typedef typename std::conditional<WIDE, int64_t, uint32_t>::type Off;
  typedef C Config;
  static constexpr bool kX = MODE == kGFwd8x, kF8 = MODE == kGFwd8 || kX, kWg = MODE == kGWgrad;
  static constexpr bool kTRows = !kWg;                          // T rows run along q
  static constexpr bool kCRows = MODE == kGFwd || kF8;
  static constexpr bool kPerm = kCRows || C::PERM;              // a lane's results: eight consecutive columns
  static constexpr int kTBytes = C::BM * 128, kCBytes = C::BN * 128;
  static constexpr int kSBytes = kF8 ? (C::BM + 63) / 64 * 256 + 256 : 0;   // scales of a step: rows, then columns / 128
  static constexpr int kStage = kTBytes + kCBytes + kSBytes;
  static constexpr int kTD = C::BM / 8 / C::W, kCD = C::BN / 8 / C::W;   // DMAs of a wave and step
  static constexpr int kThreads = C::W * 64;
  static constexpr int kIds = kWg ? 4 * 64 * 4 : 0;             // ring of row indices, 64 per step, at most three steps live
  static constexpr int kTW = (C::BM + 63) / 64, kSD = kF8 ? (kTW + C::W) / C::W : 0;   // blocks of row scales, scale DMAs of a wave

  // Byte offset, within an operand stored as 64 rows of q and R columns, of
  // the 16-byte slot holding the chunk of columns 8 c .. + 7 of row r: units
  // of 16 columns are permuted so that the eight rows half a wave reads
  // together lie in different banks.
  template <int R>
  static __device__ __forceinline__ int unit_slot(int r, int u) {
    return u ^ (((r & 3) | ((r >> 1) & 4)) & (R / 16 - 1));
  }

  // A lane's requests: `base` + `off`, step by step.
  struct Geo {
    const uint8_t* tb;
    const uint8_t* cb;
    const float* sb[kSD + 1];
    Off t[kTD], c[kCD];        // rows along q: row and chunk; else the columns' chunk
    uint32_t s[kSD + 1];
    int t_chunk, c_chunk;      // byte of the lane's chunk within a step
  };

  static __device__ __forceinline__ void request(const uint8_t* base, Off off, uint32_t lds) {
    if constexpr (WIDE) gdma16(base + off, lds);
    else gdma16s(base, off, lds);
  }

  // The swizzle of C changes with every other eight rows: only a wave alone has both kinds.
  static __device__ __forceinline__ int c_chunk_of(const Geo& g, int i) {
    return C::W % 2 && i % 2 ? g.c_chunk ^ 64 : g.c_chunk;
  }

  static __device__ __forceinline__ Geo geometry(const GroupedArgs& a, const Tile& x, int wave, int lane) {
    Geo g{};
    geometry_t(a, x, g, wave, lane);
    geometry_c(a, x, g, wave, lane);
    geometry_s(a, x, g, wave, lane);
    return g;
  }
  static __device__ __forceinline__ void geometry_t(const GroupedArgs& a, const Tile& x, Geo& g, int wave, int lane) {
    if constexpr (kTRows) {
      const bool near = !WIDE && a.t_div.div == 0;             // rows from the tile's first one
      g.tb = a.t + (near ? (int64_t)x.m0 * a.t_stride : 0);
      g.t_chunk = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
      for (int i = 0; i < kTD; ++i) {
        const int r = min(x.m0 + (wave + C::W * i) * 8 + (lane >> 3), x.hi - 1);
        const int row = max(index_row(a.t_div, a.pairs, r, a.t_rows), 0);
        g.t[i] = (Off)(near ? row - x.m0 : row) * (Off)a.t_stride + g.t_chunk;
      }
    } else {
      g.tb = a.t;
#pragma unroll
      for (int i = 0; i < kTD; ++i) {
        const int p = (wave + C::W * i) * 64 + lane, r = p / (C::BM / 8), s = p % (C::BM / 8);
        const int col = x.m0 + 16 * unit_slot<C::BM>(r, s >> 1) + 8 * (s & 1);
        g.t[i] = 2 * (col < a.M ? col : 0);
      }
    }
  }
  static __device__ __forceinline__ void geometry_c(const GroupedArgs& a, const Tile& x, Geo& g, int wave, int lane) {
    if constexpr (kCRows) {
      g.cb = a.c + (int64_t)x.e * a.c_expert + (int64_t)x.n0 * a.c_stride;
      g.c_chunk = ((lane & 7) ^ swz_c(8 * wave + (lane >> 3))) * 16;   // of block 0: c_chunk_of
#pragma unroll
      for (int i = 0; i < kCD; ++i) {
        const int n = min((wave + C::W * i) * 8 + (lane >> 3), a.N - 1 - x.n0);
        g.c[i] = (Off)n * (Off)a.c_stride + c_chunk_of(g, i);
      }
    } else {
      g.cb = a.c + (kWg ? 0 : (int64_t)x.e * a.c_expert);
#pragma unroll
      for (int i = 0; i < kCD; ++i) {
        const int p = (wave + C::W * i) * 64 + lane, r = p / (C::BN / 8), s = p % (C::BN / 8);
        const int col = x.n0 + 16 * unit_slot<C::BN>(r, s >> 1) + 8 * (s & 1);
        g.c[i] = 2 * (col < a.N ? col : 0);
      }
    }
  }
  static __device__ __forceinline__ void geometry_s(const GroupedArgs& a, const Tile& x, Geo& g, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < kSD; ++i) {
      const int b = wave + C::W * i;
      if (b < kTW) {
        const int r = x.m0 + 64 * b;
        g.sb[i] = a.t_scale + (int64_t)min(r, x.hi - 1) * a.ts_stride;
        g.s[i] = (uint32_t)max(min(lane, x.hi - 1 - r), 0) * (uint32_t)a.ts_stride * 4u;
      } else {                       // one per 128 columns of the tile, lane after lane
        const int nb = (a.N + 127) / 128, kb = (a.K + 127) / 128, n = x.n0 / 128;
        g.sb[i] = a.c_scale + ((int64_t)x.e * nb + n) * kb;
        g.s[i] = (uint32_t)min(lane, nb - 1 - n) * (uint32_t)kb * 4u;
      }
    }
  }

  // The row indices of the first N steps (kGWgrad).
  template <int N>
  static __device__ __forceinline__ void first_ids(const GroupedArgs& a, const Tile& x, uint8_t* ids, int wave, int lane) {
    for (int s = wave; s < N; s += C::W)
      reinterpret_cast<int32_t*>(ids)[s * 64 + lane] = a.pairs[min(x.lo + 64 * s + lane, x.hi - 1)];
  }

  // One request (1 KB a wave) of step j into the stage at `st`: block i of
  // this wave's share of T or C, a block of scales, the row indices.  A chunk
  // past the end of q repeats its row's first one.
  static __device__ __forceinline__ Off chunk_at(const GroupedArgs& a, int j, int chunk, Off off) {
    const int q = 128 * j;
    return q + chunk < a.K * (kF8 ? 1 : 2) ? off + (Off)q : off - (Off)chunk;
  }
  template <bool IDX>
  static __device__ __forceinline__ void issue_t(const GroupedArgs& a, const Tile& x, const Geo& g, uint32_t st,
                                                 const uint8_t* ids, int j, int i, int wave, int lane) {
    const uint32_t to = st + (wave + C::W * i) * 1024;
    if constexpr (kTRows) {
      request(g.tb, chunk_at(a, j, g.t_chunk, g.t[i]), to);
    } else {
      request_q<IDX>(a, x, a.t_div, g.tb, a.t_stride, a.t_rows, ids, j, ((wave + C::W * i) * 64 + lane) / (C::BM / 8),
                     g.t[i], to);
    }
  }
  template <bool IDX>
  static __device__ __forceinline__ void issue_c(const GroupedArgs& a, const Tile& x, const Geo& g, uint32_t st,
                                                 const uint8_t* ids, int j, int i, int wave, int lane) {
    const uint32_t to = st + kTBytes + (wave + C::W * i) * 1024;
    const int r = ((wave + C::W * i) * 64 + lane) / (C::BN / 8);
    if constexpr (kCRows) request(g.cb, chunk_at(a, j, c_chunk_of(g, i), g.c[i]), to);
    else if constexpr (kWg) request_q<IDX>(a, x, a.c_div, g.cb, a.c_stride, a.c_rows, ids, j, r, g.c[i], to);
    else request(g.cb + (int64_t)(64 * j) * a.c_stride, (Off)min(r, a.K - 1 - 64 * j) * (Off)a.c_stride + g.c[i], to);
  }
  // kGWgrad: columns `col` of the matrix row of element r of step j (the last
  // one's past the end; a row of wrong pairs is some row of the matrix).
  template <bool IDX>
  static __device__ __forceinline__ void request_q(const GroupedArgs& a, const Tile& x, const RowDiv& d,
                                                   const uint8_t* base, int64_t stride, int n_rows, const uint8_t* ids,
                                                   int j, int r, Off col, uint32_t to) {
    if (IDX && d.div != 0) {
      const int p = max(reinterpret_cast<const int32_t*>(ids)[(j & 3) * 64 + r], 0);
      request(base, (Off)min(row_of(d, p), n_rows - 1) * (Off)stride + col, to);
    } else {
      const int lo = x.lo + 64 * j;
      request(base + (int64_t)lo * stride, (Off)min(r, x.hi - 1 - lo) * (Off)stride + col, to);
    }
  }
  static __device__ __forceinline__ void issue_s(const Geo& g, uint32_t st, int j, int wave) {
#pragma unroll
    for (int i = 0; i < kSD; ++i)
      gdma4s(g.sb[i] + j, g.s[i], st + kTBytes + kCBytes + min(wave + C::W * i, kTW) * 256);
  }
  static __device__ __forceinline__ void issue_ids(const GroupedArgs& a, const Tile& x, const uint8_t* ids, int s, int lane) {
    gdma4(a.pairs + min(x.lo + 64 * (int64_t)s + lane, (int64_t)x.hi - 1), lds_addr_of(ids) + (s & 3) * 256);
  }

  // Request all of step j.
  template <bool IDX>
  static __device__ __forceinline__ void issue(const GroupedArgs& a, const Tile& x, const Geo& g, uint32_t st,
                                               const uint8_t* ids, int j, int wave, int lane) {
    if constexpr (IDX) issue_ids(a, x, ids, j + C::ST - 1, lane);   // of a later step, ahead of this step's rows
#pragma unroll
    for (int i = 0; i < kTD; ++i) issue_t<IDX>(a, x, g, st, ids, j, i, wave, lane);
#pragma unroll
    for (int i = 0; i < kCD; ++i) issue_c<IDX>(a, x, g, st, ids, j, i, wave, lane);
    issue_s(g, st, j, wave);
  }
  static constexpr int dmas(bool idx) { return kTD + kCD + kSD + (idx ? 1 : 0); }

  // Eight consecutive elements of q (half h of a step, group g of lanes) of
  // the 16 columns of unit u, from an operand stored as 64 rows of q.
  template <int R, bool PERM = false>
  static __device__ __forceinline__ uint4 read_tr(const uint8_t* base, int u, int h, int lane) {
    const int l = lane & 15, g = lane >> 4;
    uint4 v;
    uint32_t* d = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int r = 32 * h + 8 * g + 4 * p + (l >> 2);
      // PERM: units 2 p and 2 p + 1 share 32 columns, four of each eight to either
      const uint8_t* at = base + r * (2 * R) +
                          (PERM ? unit_slot<R>(r, (u & ~1) | ((l >> 1) & 1)) * 32 + (l & 1) * 16 + (u & 1) * 8
                                : unit_slot<R>(r, u) * 32 + (l & 3) * 8);
      const s16x4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4*)(uintptr_t)lds_addr_of(at));
      const uint2 w2 = __builtin_bit_cast(uint2, w);
      d[2 * p] = w2.x;
      d[2 * p + 1] = w2.y;
    }
    return v;
  }

  // The fragments of one staged step: `st` its stage, (t0, c0) the wave's
  // first 16-row and 16-column tiles; TAIL: `left` elements of q remain in
  // the step, the others are cleared.
  template <bool TAIL>
  static __device__ __forceinline__ void clear(uint4& v, int h, int g, int left) {
    if constexpr (TAIL) {
      uint32_t* d = reinterpret_cast<uint32_t*>(&v);
      const int valid = kF8 ? left - 16 * (4 * h + g) : left - 32 * h - 8 * g;
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] &= kF8 ? (valid > 0 ? 0xffffffffu : 0u) : pair_mask(valid, i);
    }
  }
  template <bool TAIL>
  static __device__ __forceinline__ uint4 read_t(const uint8_t* st, int tile, int h, int lane, int left) {
    const int l = lane & 15, g = lane >> 4;
    uint4 v;
    if constexpr (kTRows) v = *reinterpret_cast<const uint4*>(st + (16 * tile + l) * 128 + (((g + 4 * h) ^ swz_t(l)) * 16));
    else v = read_tr<C::BM>(st, tile, h, lane);
    clear<TAIL>(v, h, g, left);
    return v;
  }
  template <bool TAIL>
  static __device__ __forceinline__ uint4 read_c(const uint8_t* st, int tile, int h, int lane, int left) {
    const int l = lane & 15, g = lane >> 4;
    uint4 v;
    if constexpr (kCRows) {
      // tiles 2 p and 2 p + 1 share 32 columns: row 4 a + b of them is column 8 a + b and 8 a + 4 + b, so a lane's
      // results are eight consecutive columns
      const int row = 16 * (tile & ~1) + 8 * (l >> 2) + (l & 3) + 4 * (tile & 1);
      v = *reinterpret_cast<const uint4*>(st + kTBytes + row * 128 + (((g + 4 * h) ^ swz_c(row)) * 16));
    } else {
      v = read_tr<C::BN, C::PERM>(st + kTBytes, tile, h, lane);
    }
    clear<TAIL>(v, h, g, left);
    return v;
  }
  static __device__ __forceinline__ i32x8 join(const uint4& lo, const uint4& hi) {
    return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  }
  static __device__ __forceinline__ const float* scales(const uint8_t* st) {
    return reinterpret_cast<const float*>(st + kTBytes + kCBytes);
  }

  // Multiply one staged step into the accumulators.
  template <bool TAIL>
  static __device__ __forceinline__ void compute(const uint8_t* st, int wm, int wn, int lane, int left,
                                                 f32x4 (&acc)[C::CT][C::TT]) {
    const int l = lane & 15;
    const int t0 = wm * C::TT, c0 = wn * C::CT;
    if constexpr (kF8) {
      const float* sc = scales(st);
      float ts[C::TT], cs[C::CT];
      i32x8 cv[C::CT];
#pragma unroll
      for (int i = 0; i < C::CT; ++i) {
        cv[i] = join(read_c<TAIL>(st, c0 + i, 0, lane, left), read_c<TAIL>(st, c0 + i, 1, lane, left));
        cs[i] = sc[64 * kTW + (c0 + i) / 8];
      }
#pragma unroll
      for (int j = 0; j < C::TT; ++j) ts[j] = sc[16 * (t0 + j) + l];
      // multiply-adds two MFMAs behind, as in phase_mul
      constexpr int kN = C::TT * C::CT, kBehind = kX ? 0 : 2;
      f32x4 p[kN];
      i32x8 tv;
#pragma unroll
      for (int q = 0; q < kN + kBehind; ++q) {
        if (q < kN) {
          const int j = q / C::CT, i = q % C::CT;
          if (i == 0) tv = join(read_t<TAIL>(st, t0 + j, 0, lane, left), read_t<TAIL>(st, t0 + j, 1, lane, left));
          p[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          if constexpr (kX) {
#pragma unroll
            for (int h = 0; h < 4; ++h)
              p[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8x8_to_bf16x8(cv[i][2 * h], cv[i][2 * h + 1]),
                                                             fp8x8_to_bf16x8(tv[2 * h], tv[2 * h + 1]), p[q], 0, 0, 0);
          } else {
            p[q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(cv[i], tv, p[q], 0, 0, 0, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        if (q >= kBehind) {
          const int r = q - kBehind, j = r / C::CT, i = r % C::CT;
          const float s = ts[j] * cs[i];
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][j][k] = fmaf(p[r][k], s, acc[i][j][k]);
          if constexpr (!kX) __builtin_amdgcn_sched_barrier(0);
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bf16x8 cv[C::CT];
#pragma unroll
        for (int i = 0; i < C::CT; ++i) cv[i] = __builtin_bit_cast(bf16x8, read_c<TAIL>(st, c0 + i, h, lane, left));
#pragma unroll
        for (int j = 0; j < C::TT; ++j) {
          const bf16x8 tv = __builtin_bit_cast(bf16x8, read_t<TAIL>(st, t0 + j, h, lane, left));
#pragma unroll
          for (int i = 0; i < C::CT; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cv[i], tv, acc[i][j], 0, 0, 0);
        }
      }
    }
  }

  // The same step in four phases for two groups of waves taking turns (see
  // grouped_pair_kernel).  The column fragments of a half of the step stay in
  // registers until their second phase; row fragments are read for each.
  //   E4M3             phase p: quarter p of the rows, all of the step
  //   T rows along q   phase p: half p / 2 of the rows, half p % 2 of the step
  //   T rows along t   phase p: half p % 2 of the rows, half p / 2 of the step
  static constexpr int kRowsOf(int p) { return kTRows ? p / 2 : p % 2; }
  static constexpr int kHalfOf(int p) { return kTRows ? p % 2 : p / 2; }
  struct Phase {
    uint4 c[C::CT][2], t[C::TT / 2];
    float ts[C::TT / 4 + 1], cs;
  };
  template <int P, bool TAIL>
  static __device__ __forceinline__ void phase_read(const uint8_t* st, int wm, int wn, int lane, int left, Phase& f) {
    const int t0 = wm * C::TT, c0 = wn * C::CT;
    if constexpr (kF8) {
      if constexpr (P == 0) {
#pragma unroll
        for (int i = 0; i < C::CT; ++i) {
          f.c[i][0] = read_c<TAIL>(st, c0 + i, 0, lane, left);
          f.c[i][1] = read_c<TAIL>(st, c0 + i, 1, lane, left);
        }
        f.cs = scales(st)[64 * kTW + c0 / 8];
      }
#pragma unroll
      for (int j = 0; j < C::TT / 4; ++j) {
        f.t[2 * j] = read_t<TAIL>(st, t0 + P * (C::TT / 4) + j, 0, lane, left);
        f.t[2 * j + 1] = read_t<TAIL>(st, t0 + P * (C::TT / 4) + j, 1, lane, left);
        f.ts[j] = scales(st)[16 * (t0 + P * (C::TT / 4) + j) + (lane & 15)];
      }
    } else {
      constexpr int H = kHalfOf(P);
      if constexpr (P == 0 || H != kHalfOf(P - 1)) {
        if constexpr (kTRows ? P < 2 : true) {
#pragma unroll
          for (int i = 0; i < C::CT; ++i) f.c[i][kTRows ? H : 0] = read_c<TAIL>(st, c0 + i, H, lane, left);
        }
      }
#pragma unroll
      for (int j = 0; j < C::TT / 2; ++j)
        f.t[j] = read_t<TAIL>(st, t0 + kRowsOf(P) * (C::TT / 2) + j, H, lane, left);
    }
  }
  template <int P>
  static __device__ __forceinline__ void phase_mul(const Phase& f, f32x4 (&acc)[C::CT][C::TT]) {
    if constexpr (kF8) {
      // an MFMA takes 32 cycles, its four multiply-adds 16 and must wait for it: they are held two MFMAs behind
      constexpr int kN = C::TT / 4 * C::CT, kBehind = 2;
      f32x4 p[kN];
      float s[C::TT / 4];
#pragma unroll
      for (int j = 0; j < C::TT / 4; ++j) s[j] = f.ts[j] * f.cs;
#pragma unroll
      for (int q = 0; q < kN + kBehind; ++q) {
        if (q < kN) {
          const int j = q / C::CT, i = q % C::CT;
          const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
          p[q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(f.c[i][0], f.c[i][1]),
                                                                  join(f.t[2 * j], f.t[2 * j + 1]), z, 0, 0, 0, 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (q >= kBehind) {
          const int r = q - kBehind, j = r / C::CT, i = r % C::CT;
          f32x4& d = acc[i][P * (C::TT / 4) + j];
#pragma unroll
          for (int k = 0; k < 4; ++k) d[k] = fmaf(p[r][k], s[j], d[k]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < C::TT / 2; ++j)
#pragma unroll
        for (int i = 0; i < C::CT; ++i) {
          f32x4& d = acc[i][kRowsOf(P) * (C::TT / 2) + j];
          d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f.c[i][kTRows ? kHalfOf(P) : 0]),
                                                      __builtin_bit_cast(bf16x8, f.t[j]), d, 0, 0, 0);
        }
    }
  }

  // The requests of a step, in four groups of two or three per wave, in the
  // order they are made and needed (grouped_pair_kernel):
  //   T rows along q: C (0, 1), C (2, 3), T of the first half of the rows with
  //     the scales, T of the second;
  //   T rows along t: T and C of the first half of the step, T and C of the second.
  static constexpr int kGroup[4] = {2, 2, 2 + kSD, 2};
  template <int G, bool IDX>
  static __device__ __forceinline__ void issue_group(const GroupedArgs& a, const Tile& x, const Geo& g, uint32_t lds0,
                                                     const uint8_t* ids, int j, int wave, int lane) {
    const uint32_t st = lds0 + (j & 1) * kStage;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (kTRows) {
        if constexpr (G < 2) issue_c<IDX>(a, x, g, st, ids, j, 2 * G + i, wave, lane);
        else issue_t<IDX>(a, x, g, st, ids, j, (G - 2) + 2 * i, wave, lane);
      } else {
        if constexpr (G % 2 == 0) issue_t<IDX>(a, x, g, st, ids, j, G + i, wave, lane);
        else issue_c<IDX>(a, x, g, st, ids, j, G - 1 + i, wave, lane);
      }
    }
    if constexpr (G == 2) issue_s(g, st, j, wave);
  }

  // Whether none of the wave's rows or columns are stored: it then makes its
  // requests and keeps the barriers, but leaves the LDS and the matrix cores
  // to the others.  A group's last tile is half empty on average: 16384 rows in
  // 104 of 112 groups, 1536 x 3584 E4M3, 212 us without this and 196 with it, timed
  // in turn on one card (185 to 190 on others).
  static __device__ __forceinline__ bool idle(const GroupedArgs& a, const Tile& x, int wm, int wn) {
    return x.m0 + 16 * wm * C::TT >= (kWg ? a.M : x.hi) || x.n0 + 16 * wn * C::CT >= a.N;
  }

  // Where row tile j (of the workgroup's tile) goes in this lane; null if nowhere.
  static __device__ __forceinline__ uint8_t* out_row(const GroupedArgs& a, const Tile& x, int j, int lane) {
    const int t = x.m0 + 16 * j + (lane & 15);
    if (t >= (kWg ? a.M : x.hi)) return nullptr;
    const int row = kWg ? t : index_row(a.o_div, a.pairs, t, a.o_rows);
    if (row < 0) return nullptr;
    return static_cast<uint8_t*>(a.out) + (kWg ? (int64_t)x.e * a.out_expert : 0) + (int64_t)row * a.out_stride;
  }
  // The first of the four columns of column tile i that this lane holds.
  static __device__ __forceinline__ int out_col(const Tile& x, int i, int lane) {
    const int g = lane >> 4;
    return x.n0 + (kPerm ? 16 * (i & ~1) + 8 * g + 4 * (i & 1) : 16 * i + 4 * g);
  }
  // Where the wave's row tiles go, all looked up before the first store.
  static __device__ __forceinline__ void out_rows(const GroupedArgs& a, const Tile& x, int wm, int lane,
                                                  uint8_t* (&o)[C::TT]) {
#pragma unroll
    for (int j = 0; j < C::TT; ++j) o[j] = out_row(a, x, wm * C::TT + j, lane);
  }
  // Store the wave's tile.  A lane has 16 bytes of a row at a time (four fp32 or
  // eight bf16), four lanes 64 bytes in a row; lanes 2 i and 2 i + 1 exchange
  // halves of two such units so that eight lanes store a row's 128, whole
  // lines (dw of 8191 rows x 1536 x 3584 in fp32: 246 us without, 222 with it).
  static __device__ __forceinline__ void epilogue(const GroupedArgs& a, const Tile& x, int wn, int lane,
                                                  uint8_t* const (&o)[C::TT], f32x4 (&acc)[C::CT][C::TT]) {
    const bool odd = lane & 1;
#pragma unroll
    for (int j = 0; j < C::TT; ++j) {
      const uint64_t own = (uint64_t)o[j];
      const uint64_t other = (uint64_t)swap_pair((uint32_t)own) | (uint64_t)swap_pair((uint32_t)(own >> 32)) << 32;
      uint8_t* even_row = reinterpret_cast<uint8_t*>(odd ? other : own);
      uint8_t* odd_row = reinterpret_cast<uint8_t*>(odd ? own : other);
      if (a.out_f32) {
#pragma unroll
        for (int i = 0; i < C::CT; i += 2) {
          const uint4 u = __builtin_bit_cast(uint4, acc[i][j]), v = __builtin_bit_cast(uint4, acc[i + 1][j]);
          const uint4 got = swap_pair(pick(odd, u, v));
          const int col = out_col(x, wn * C::CT + i + (odd ? 1 : 0), lane);
          if (even_row) store4(a, even_row, col, __builtin_bit_cast(f32x4, pick(odd, got, u)));
          if (odd_row) store4(a, odd_row, col, __builtin_bit_cast(f32x4, pick(odd, v, got)));
        }
      } else if constexpr (kPerm && C::CT % 4 == 0) {
#pragma unroll
        for (int i = 0; i < C::CT; i += 4) {
          const uint4 u = pack8(acc[i][j], acc[i + 1][j]), v = pack8(acc[i + 2][j], acc[i + 3][j]);
          const uint4 got = swap_pair(pick(odd, u, v));
          const int col = out_col(x, wn * C::CT + i + (odd ? 2 : 0), lane);
          if (even_row) store8(a, even_row, col, pick(odd, got, u));
          if (odd_row) store8(a, odd_row, col, pick(odd, v, got));
        }
      } else if (o[j]) {
#pragma unroll
        for (int i = 0; i < C::CT; i += 2) {
          if constexpr (kPerm) {
            store8(a, o[j], out_col(x, wn * C::CT + i, lane), pack8(acc[i][j], acc[i + 1][j]));
          } else {
            store4(a, o[j], out_col(x, wn * C::CT + i, lane), acc[i][j]);
            store4(a, o[j], out_col(x, wn * C::CT + i + 1, lane), acc[i + 1][j]);
          }
        }
      }
    }
  }
};

// The groups of a launch, kept in LDS (a second array would cost Mid and Short
// a workgroup a CU): the exclusive prefix of their row tiles (of BM rows), or
// (kGWgrad) where each begins.
struct Table {
  int at[kMaxE + 1], part[16];
};

template <int NT, int BM, bool FIRST>
__device__ __forceinline__ void make_table(const GroupedArgs& a, Table& t, int tid) {
  constexpr int kPer = kMaxE / NT;
  int at_e[kPer + 1];
#pragma unroll
  for (int i = 0; i <= kPer; ++i) at_e[i] = min(max(a.offsets[min(tid * kPer + i, a.experts)], 0), a.rows);
  if constexpr (FIRST) {
#pragma unroll
    for (int i = 0; i <= kPer; ++i)
      if (tid * kPer + i <= a.experts) t.at[tid * kPer + i] = at_e[i];
    __syncthreads();
    return;
  }
  int cnt[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    cnt[i] = tid * kPer + i < a.experts ? (max(at_e[i + 1] - at_e[i], 0) + BM - 1) / BM : 0;
    sum += cnt[i];
  }
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int up = __shfl_up(inc, d, kWave);
    if ((tid & 63) >= d) inc += up;
  }
  if ((tid & 63) == 63) t.part[tid >> 6] = inc;
  __syncthreads();
  int at = inc - sum;
  for (int w = 0; w < (tid >> 6); ++w) at += t.part[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (tid * kPer + i <= a.experts) t.at[tid * kPer + i] = at;
    at += cnt[i];
  }
  if (tid == NT - 1 && a.experts == kMaxE) t.at[kMaxE] = at;
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

// A workgroup barrier that neither waits for memory nor lets anything move
// across it.
__device__ __forceinline__ void part_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
// Wait until this wave's requests but the last N have landed.  They complete in
// the order issued, so a store or a spilled register among them can only make
// the wait longer.
template <int N>
__device__ __forceinline__ void land() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
template <class K, int P, class A>
__device__ __forceinline__ void phase_mul_fenced(const typename K::Phase& f, A& acc) {
  __builtin_amdgcn_s_setprio(1);
  K::template phase_mul<P>(f, acc);
  __builtin_amdgcn_s_setprio(0);
  part_barrier();
}

// The tiles of one workgroup, in order.
template <class K>
struct Walk {
  using C = typename K::Config;
  int m_tiles, slots, it, last;      // launch_as keeps the number of tiles below 2^31

  template <int NT>
  __device__ __forceinline__ Walk(const GroupedArgs& a, Table& t, int tid, std::integral_constant<int, NT>) {
    if (a.offsets) make_table<NT, C::BM, K::kWg>(a, t, tid);
    if constexpr (K::kWg) {
      m_tiles = a.experts * a.m_bound;
    } else if (a.offsets) {
      m_tiles = min(t.at[a.experts], a.m_bound);   // ascending offsets never exceed the bound
    } else {
      m_tiles = a.m_bound;
    }
    // each XCD (workgroups b, b + 8, ...) walks a contiguous share of the tiles
    const int64_t total = (int64_t)m_tiles * a.n_tiles;
    const int xcds = min((int)gridDim.x, 8), xcd = blockIdx.x % xcds;
    slots = gridDim.x / xcds;
    it = (int)(total * xcd / xcds) + blockIdx.x / xcds;
    last = (int)(total * (xcd + 1) / xcds);
  }

  // Moves on to the next tile that holds something; false if there is none.
  __device__ __forceinline__ bool next(const GroupedArgs& a, const Table& t, int lane, Tile& x, int& steps, int& left) {
    for (; it < last; it += slots) {
      if (tile(a, t, lane, x, steps, left)) {
        it += slots;
        return true;
      }
    }
    return false;
  }

  // The tile `it`; false if it holds nothing (only with offsets that do not ascend).
  __device__ __forceinline__ bool tile(const GroupedArgs& a, const Table& t, int lane, Tile& x, int& steps, int& left) {
    if constexpr (K::kWg) {
      const int per = a.m_bound * a.n_tiles;
      x.e = it / per;
      const int r = it - x.e * per;
      x.m0 = (r % a.m_bound) * C::BM;
      x.n0 = (r / a.m_bound) * C::BN;
      x.lo = a.offsets ? t.at[x.e] : 0;
      x.hi = a.offsets ? max(t.at[x.e + 1], x.lo) : a.rows;
      steps = (x.hi - x.lo + 63) / 64;
      left = x.hi - x.lo - 64 * (steps - 1);
      return true;
    } else {
      // within a group: eight row tiles by all column tiles, rows fastest
      int local, m_l;
      if (a.offsets) {
        x.e = __builtin_amdgcn_readfirstlane(find_group(t.at, a.experts, it / a.n_tiles, lane));
        local = it - t.at[x.e] * a.n_tiles;
        m_l = t.at[x.e + 1] - t.at[x.e];
      } else {
        x.e = 0;
        local = it;
        m_l = m_tiles;
      }
      group_rows(a, x.e, x.lo, x.hi);
      const int block = local / (8 * a.n_tiles), in = local % (8 * a.n_tiles);
      const int high = min(8, m_l - 8 * block);
      x.m0 = x.lo + (8 * block + in % high) * C::BM;
      x.n0 = (in / high) * C::BN;
      constexpr int kQ = K::kF8 ? 128 : 64;
      steps = (a.K + kQ - 1) / kQ;
      left = a.K - kQ * (steps - 1);
      return x.m0 < x.hi && x.n0 < a.N;
    }
  }
};

template <class C, int MODE, bool IDX>
__global__ __launch_bounds__(C::W * 64, C::MINB) void grouped_kernel(GroupedArgs a) {
  using K = Kernel<C, MODE, true>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::ST * K::kStage + K::kIds + sizeof(Table)];
  uint8_t* ids = lds + C::ST * K::kStage;
  Table& table = *reinterpret_cast<Table*>(lds + C::ST * K::kStage + K::kIds);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const uint32_t lds0 = lds_addr_of(lds);

  Walk<K> w(a, table, tid, std::integral_constant<int, K::kThreads>{});
  Tile x;
  int steps, left;
  typename K::Geo g;
  // go on to the next tile that holds something and request its first steps
  auto start = [&]() {
    if (!w.next(a, table, lane, x, steps, left)) return false;
    if (steps == 0) return true;
    g = K::geometry(a, x, wave, lane);
    if constexpr (IDX) {
      K::template first_ids<C::ST - 1>(a, x, ids, wave, lane);
      __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < C::ST - 1; ++s)
      if (s < steps) K::template issue<IDX>(a, x, g, lds0 + s * K::kStage, ids, s, wave, lane);
    return true;
  };

  bool more = start();
  while (more) {
    const bool tail = left < (K::kF8 ? 128 : 64), idle = K::idle(a, x, wm, wn);
    f32x4 acc[C::CT][C::TT];
#pragma unroll
    for (int i = 0; i < C::CT; ++i)
#pragma unroll
      for (int j = 0; j < C::TT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

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
      else if (!idle) K::template compute<false>(st, wm, wn, lane, left, acc);
      stage = stage + 1 == C::ST ? 0 : stage + 1;
    }
    lds_barrier();                                           // all fragments of the tile have been read
    const Tile done = x;
    more = start();                                          // under way while the results are stored
    uint8_t* o[C::TT];
    K::out_rows(a, done, wm, lane, o);
    K::epilogue(a, done, wn, lane, o, acc);
  }
}

// Few tiles, long contractions: the waves of a workgroup split q between them,
// wave w taking steps w, w + KS, ... of the same tile with stages of its own,
// so there is no barrier in the loop; the partial sums are added in LDS in the
// waves' order.  With one tile a CU the kernel above spends 0.45 us on a step
// of 64 x 64 (barrier, requests, LDS and MFMA latency in turn); here KS steps
// are under way at once.
template <class C, int MODE, int KS>
__global__ __launch_bounds__(KS * 64, 1) void grouped_split_kernel(GroupedArgs a) {
  using K = Kernel<C, MODE, true>;
  static_assert(C::W == 1, "a wave computes the whole tile");
  constexpr int kStages = KS * C::ST * K::kStage, kSums = KS * C::CT * C::TT * 1024;
  static_assert(kSums <= kStages, "the sums fit the stages");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kStages + sizeof(Table)];
  Table& table = *reinterpret_cast<Table*>(lds + kStages);
  const int tid = threadIdx.x, lane = tid & 63, wk = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint8_t* own = lds + wk * C::ST * K::kStage;
  const uint32_t own0 = lds_addr_of(own);
  f32x4* sums = reinterpret_cast<f32x4*>(lds);
  constexpr int kD = K::dmas(false);

  Walk<K> w(a, table, tid, std::integral_constant<int, KS * 64>{});
  Tile x;
  int steps, left;
  while (w.next(a, table, lane, x, steps, left)) {
    f32x4 acc[C::CT][C::TT];
#pragma unroll
    for (int i = 0; i < C::CT; ++i)
#pragma unroll
      for (int j = 0; j < C::TT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int mine = wk < steps ? (steps - wk + KS - 1) / KS : 0;   // steps of this wave
    if (mine > 0) {
      const typename K::Geo g = K::geometry(a, x, 0, lane);
#pragma unroll
      for (int s = 0; s < C::ST - 1; ++s)
        if (s < mine) K::template issue<false>(a, x, g, own0 + s * K::kStage, nullptr, wk + s * KS, 0, lane);
      int stage = 0;
      for (int u = 0; u < mine; ++u) {
        const int j = wk + u * KS;
        const int ahead = stage == 0 ? C::ST - 1 : stage - 1;
        // the stage ahead was read a step ago, and its fragments have arrived
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (u + C::ST - 1 < mine) {
          K::template issue<false>(a, x, g, own0 + ahead * K::kStage, nullptr, j + (C::ST - 1) * KS, 0, lane);
          land<(C::ST - 1) * kD>();
        } else {
          land<0>();
        }
        const uint8_t* st = own + stage * K::kStage;
        if (j == steps - 1) K::template compute<true>(st, 0, 0, lane, left, acc);
        else K::template compute<false>(st, 0, 0, lane, left, acc);
        stage = stage + 1 == C::ST ? 0 : stage + 1;
      }
    }
    __syncthreads();                               // the stages have been read
#pragma unroll
    for (int i = 0; i < C::CT; ++i)
#pragma unroll
      for (int j = 0; j < C::TT; ++j) sums[((wk * C::CT + i) * C::TT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int q = wk; q < C::CT * C::TT; q += KS) {
      const int i = q / C::TT, j = q % C::TT;
      uint8_t* o = K::out_row(a, x, j, lane);
      if (!o) continue;
      f32x4 v = sums[q * 64 + lane];
#pragma unroll
      for (int s = 1; s < KS; ++s) v += sums[(s * C::CT * C::TT + q) * 64 + lane];
      store4(a, o, K::out_col(x, i, lane), v);
    }
    __syncthreads();                               // the sums have been read
  }
}

// Contractions of one step (bf16, 64 elements: adapters' ranks): the time is
// the output's.  A workgroup owns 128 columns of one group, keeps their
// fragments in registers and walks every a.m_bound-th tile of 64 rows, two
// tiles requested ahead of the stores.  The group comes from the block index,
// so there is no table to build.  16384 rows x 768 x 32: 20 us in grouped_kernel,
// 15.6 here at first and 12.8 with later steps (whole-line stores past the
// caches); input gradient 8192 x 3584 x 32: 39, 31 and 19 us (4.5 TB/s).
template <class C, int MODE>
__global__ __launch_bounds__(256, 4) void grouped_thin_kernel(GroupedArgs a) {
  using K = Kernel<C, MODE, true>;
  static_assert(C::W == 4 && C::ST == 3 && K::kTRows && !K::kF8, "bf16 rows along q, three row stages");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::ST * K::kTBytes + K::kCBytes];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  // T stage s lies at s * kTBytes, so C, which issue_c and read_c put kTBytes
  // behind a stage, behind the last one
  const uint8_t* last = lds + (C::ST - 1) * K::kTBytes;
  Tile x;
  x.e = blockIdx.x / (a.n_tiles * a.m_bound);
  const int in = blockIdx.x % (a.n_tiles * a.m_bound);
  x.n0 = (in % a.n_tiles) * C::BN;
  group_rows(a, x.e, x.lo, x.hi);
  const int first = x.lo + in / a.n_tiles * C::BM, stride = a.m_bound * C::BM;
  if (first >= x.hi) return;
  const int tiles = (x.hi - first + stride - 1) / stride;

  typename K::Geo g{};
  K::geometry_c(a, x, g, wave, lane);
#pragma unroll
  for (int i = 0; i < K::kCD; ++i) K::template issue_c<false>(a, x, g, lds_addr_of(last), nullptr, 0, i, wave, lane);
  auto request_rows = [&](int u) {
    Tile y = x;
    y.m0 = first + u * stride;
    K::geometry_t(a, y, g, wave, lane);
#pragma unroll
    for (int i = 0; i < K::kTD; ++i)
      K::template issue_t<false>(a, y, g, lds_addr_of(lds) + u % C::ST * K::kTBytes, nullptr, 0, i, wave, lane);
  };
  request_rows(0);
  if (tiles > 1) request_rows(1);
  if (tiles > 1) dma_barrier<K::kTD>();
  else dma_barrier<0>();
  bf16x8 cv[C::CT][2];
#pragma unroll
  for (int i = 0; i < C::CT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      cv[i][h] = __builtin_bit_cast(bf16x8, K::template read_c<true>(last, wn * C::CT + i, h, lane, a.K));
  for (int u = 0; u < tiles; ++u) {
    if (u > 0) dma_barrier<0>();                   // this tile's rows; the last tile's stores are long under way
    Tile y = x;
    y.m0 = first + u * stride;
    uint8_t* o[C::TT];
    K::out_rows(a, y, wm, lane, o);
    if (u + 2 < tiles) request_rows(u + 2);        // into the stage read a tile ago
    f32x4 acc[C::CT][C::TT];
    const uint8_t* st = lds + u % C::ST * K::kTBytes;
#pragma unroll
    for (int j = 0; j < C::TT; ++j) {
      bf16x8 tv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        tv[h] = __builtin_bit_cast(bf16x8, K::template read_t<true>(st, wm * C::TT + j, h, lane, a.K));
#pragma unroll
      for (int i = 0; i < C::CT; ++i) {
        const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cv[i][0], tv[0], z, 0, 0, 0);
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(cv[i][1], tv[1], acc[i][j], 0, 0, 0);
      }
    }
    K::epilogue(a, x, wn, lane, o, acc);
  }
}

// Large tiles: two groups of four waves, one wave of each on every SIMD, take
// turns.  A step has four phases, each a reading part R (fragments from LDS,
// requests for later steps) and a multiplying part M (1/4 of the step's
// MFMAs), with a workgroup barrier after every part; the second group runs
// one part behind, so that while one group multiplies the other reads.
//
// Two stages hold steps j and j + 1, and a region is requested again as soon
// as its step has been read, so that requests have about a step to land
// (issue_group's groups 0 .. 3):
//   R3(j): group 0 of step j + 2     R1(j): group 2 of step j + 1
//   R0(j): group 1 of step j + 1     R2(j): group 3 of step j + 1
// Regions: groups 0 and 1 are last read in R1, group 2 in R1 (T rows along q)
// or R2 to R3, group 3 in R3, and the scales in R3.  A fragment read in Rk
// is in its register by the end of Mk.  The first group issues one part ahead
// of the second: its R(k + 2) begins when the second group's M(k) has ended.
// Group 0 in R3 overwrites what R1 read, group 1 in R0 and group 2 in R1 of the
// next step what R1 and R3 read: two parts R on, or more.  Group 3 in R2 is
// three parts R after R3.
// Landing: R0 of a step needs its groups 0 to 2 (T rows along t: 0 and 1), R2 the
// rest.  Each wave waits for its own requests before the barrier that ends R3
// (or R1); the first group begins R0 (R2) at the barrier that ends the second
// group's R3 (R1), so by then every wave has waited.
//
// A step (256 x 256 x 64 bf16) takes 1.18 us with one tile on the chip, 0.89
// without its requests, and 1.55 with all of them in R0, waited for in R3 (4096
// x 4096 x 16384: 455 us against 523).  With all CUs busy it takes 1.75 (E4M3,
// 128 deep, 2.0), and 1.42 to 1.58 without requests.  The matrix cores are busy
// 65 % of the forward kernel's time in bf16 and 52 % in E4M3, so no one thing is
// the bound: requests are a fifth of a step, and the reading parts' barriers and
// waits, the rounds' last tiles and the stores the rest.  8192 x 7168 x 3584
// E4M3: 217 and 249 us on two cards (1.94 and 1.69 PFLOP/s), whose clocks under
// this load differ.
template <class C, int MODE, bool IDX>
__global__ __launch_bounds__(512, 2) void grouped_pair_kernel(GroupedArgs a) {
  using K = Kernel<C, MODE, false>;
  static_assert(C::W == 8 && C::ST == 2 && C::TT % 4 == 0 && K::kTD == 4 && K::kCD == 4,
                "two groups of four waves, two stages, four phases, groups of two requests");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * K::kStage + K::kIds + sizeof(Table)];
  uint8_t* ids = lds + 2 * K::kStage;
  Table& table = *reinterpret_cast<Table*>(lds + 2 * K::kStage + K::kIds);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const uint32_t lds0 = lds_addr_of(lds);
  // requests made after those waited for, up to the wait (the row indices of
  // step j + 3 go with R1): in R3 for groups 0 .. 2 (0 .. 1) of the next step,
  // in R1 for the rest of this one
  constexpr int kI = IDX ? 1 : 0;
  constexpr int kAfterR3 = K::kTRows ? K::kGroup[3] + K::kGroup[0]
                                     : K::kGroup[2] + kI + K::kGroup[3] + K::kGroup[0];
  constexpr int kAfterR1 = K::kGroup[0] + K::kGroup[1] + K::kGroup[2] + kI;

  Walk<K> w(a, table, tid, std::integral_constant<int, K::kThreads>{});
  Tile x;
  int steps, left;
  typename K::Geo g;
  // go on to the next tile that holds something and request its first step
  auto start = [&]() {
    if (!w.next(a, table, lane, x, steps, left)) return false;
    if (steps == 0) return true;
    g = K::geometry(a, x, wave, lane);
    if constexpr (IDX) {
      K::template first_ids<3>(a, x, ids, wave, lane);
      __syncthreads();
    }
    K::template issue_group<0, IDX>(a, x, g, lds0, ids, 0, wave, lane);
    K::template issue_group<1, IDX>(a, x, g, lds0, ids, 0, wave, lane);
    K::template issue_group<2, IDX>(a, x, g, lds0, ids, 0, wave, lane);
    K::template issue_group<3, IDX>(a, x, g, lds0, ids, 0, wave, lane);
    if (steps > 1) K::template issue_group<0, IDX>(a, x, g, lds0, ids, 1, wave, lane);
    return true;
  };

  bool more = start();
  while (more) {
    f32x4 acc[C::CT][C::TT];
#pragma unroll
    for (int i = 0; i < C::CT; ++i)
#pragma unroll
      for (int j = 0; j < C::TT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    if (steps > 0) {
      dma_barrier<0>();
      if (wave >= 4) part_barrier();
      typename K::Phase f;
      // AHEAD: steps that follow, 2 for two or more; the last step may end inside
      auto step = [&](auto ahead, auto works, int j) {
        constexpr int kA = decltype(ahead)::value;
        constexpr bool kT = kA == 0, kWorks = decltype(works)::value;
        const uint8_t* st = lds + (j & 1) * K::kStage;
        if constexpr (kWorks) K::template phase_read<0, kT>(st, wm, wn, lane, left, f);
        if constexpr (kA > 0) K::template issue_group<1, IDX>(a, x, g, lds0, ids, j + 1, wave, lane);
        part_barrier();
        if constexpr (kWorks) phase_mul_fenced<K, 0>(f, acc);
        else part_barrier();
        if constexpr (kWorks) K::template phase_read<1, kT>(st, wm, wn, lane, left, f);
        if constexpr (kA > 0) {
          if constexpr (IDX) K::issue_ids(a, x, ids, j + 3, lane);
          K::template issue_group<2, IDX>(a, x, g, lds0, ids, j + 1, wave, lane);
          land<kAfterR1>();
        } else {
          land<0>();
        }
        part_barrier();
        if constexpr (kWorks) phase_mul_fenced<K, 1>(f, acc);
        else part_barrier();
        if constexpr (kWorks) K::template phase_read<2, kT>(st, wm, wn, lane, left, f);
        if constexpr (kA > 0) K::template issue_group<3, IDX>(a, x, g, lds0, ids, j + 1, wave, lane);
        part_barrier();
        if constexpr (kWorks) phase_mul_fenced<K, 2>(f, acc);
        else part_barrier();
        if constexpr (kWorks) K::template phase_read<3, kT>(st, wm, wn, lane, left, f);
        if constexpr (kA > 1) {
          K::template issue_group<0, IDX>(a, x, g, lds0, ids, j + 2, wave, lane);
          land<kAfterR3>();
        } else {
          land<0>();
        }
        part_barrier();
        if constexpr (kWorks) phase_mul_fenced<K, 3>(f, acc);
        else part_barrier();
      };
      auto all = [&](auto works) {
        for (int j = 0; j < steps - 2; ++j) step(std::integral_constant<int, 2>{}, works, j);
        if (steps > 1) step(std::integral_constant<int, 1>{}, works, steps - 2);
        step(std::integral_constant<int, 0>{}, works, steps - 1);
      };
      if (K::idle(a, x, wm, wn)) all(std::false_type{});
      else all(std::true_type{});
      if (wave < 4) part_barrier();                          // all fragments of the tile have been read
    }
    const Tile done = x;
    more = start();                                          // under way while the results are stored
    uint8_t* o[C::TT];
    K::out_rows(a, done, wm, lane, o);
    K::epilogue(a, done, wn, lane, o, acc);
  }
}

// As many workgroups as the chip holds, so long as a group's share of the rows
// has tiles for them.  The share is the mean: 16384 rows x 768 x 32 in 112 groups
// take 10 us, with half of the rows in one group 62, with all in one 120.
template <class C, int MODE>
hipError_t launch_thin(GroupedArgs& a, int cus, hipStream_t s) {
  a.n_tiles = (a.N + C::BN - 1) / C::BN;
  const int64_t columns = (int64_t)a.n_tiles * a.experts, rows = (a.rows / a.experts + C::BM - 1) / C::BM + 1;
  a.m_bound = (int32_t)std::max<int64_t>(1, std::min((4 * (int64_t)cus + columns - 1) / columns, rows));
  hipLaunchKernelGGL((grouped_thin_kernel<C, MODE>), dim3((unsigned)(columns * a.m_bound)), dim3(256), 0, s, a);
  return hipGetLastError();
}

// KS: waves that split q (grouped_split_kernel); 0: grouped_kernel, -1: grouped_pair_kernel.
template <class C, int MODE, bool IDX, int KS = 0>
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
  if (tiles >= (int64_t)1 << 31) return hipErrorInvalidValue;   // beyond any memory: 2^31 tiles of 2^11 results or more
  const int64_t most = KS > 0 ? cus : (int64_t)C::MINB * 4 / C::W * cus;   // resident workgroups
  int64_t grid = tiles < most ? tiles : most;
  if (grid > 8) grid = (grid + 7) / 8 * 8;
  if constexpr (KS > 0) hipLaunchKernelGGL((grouped_split_kernel<C, MODE, KS>), dim3((unsigned)grid), dim3(KS * 64), 0, s, a);
  else if constexpr (KS < 0) hipLaunchKernelGGL((grouped_pair_kernel<C, MODE, IDX>), dim3((unsigned)grid), dim3(512), 0, s, a);
  else hipLaunchKernelGGL((grouped_kernel<C, MODE, IDX>), dim3((unsigned)grid), dim3(C::W * 64), 0, s, a);
  return hipGetLastError();
}

// Whether 32-bit offsets reach every row a tile of grouped_pair_kernel reads
// (Kernel's WIDE): gathered rows from the start of their array, others from the
// tile's first row (a step's 64, or the tile's 256).
bool narrow_ok(GroupedMode mode, const GroupedArgs& a) {
  const int64_t lim = (int64_t)1 << 32;
  const auto fits = [&](const RowDiv& d, int64_t stride, int32_t rows) {
    return (d.div && a.pairs ? (int64_t)rows : 256) * stride < lim;
  };
  if (!fits(a.t_div, a.t_stride, a.t_rows)) return false;
  if (mode == kGWgrad && !fits(a.c_div, a.c_stride, a.c_rows)) return false;
  return 256 * a.c_stride < lim && 256 * a.ts_stride * 4 < lim;
}

// The tile shape: the one whose rounds over the chip cost least, a round being
// steps * (time of a step) + (first requests and last stores).  Times in us on
// an MI355X, with one workgroup a CU and with all that fit (kCosts): fitted to
// single rounds (64 rows) and many (8192 rows), k 3584 to 7168.  So measured,
// with 3584 columns and k 3584 (Small / Mid / Large / Pair):
//   bf16   64 rows 28 / 32 / 44 / 68 us,  1024 rows 63 / 45 / 50 / 77,
//          2048 rows 113 / 80 / 66 / 81,  4096 rows 208 / 147 / 133 / 96
//   E4M3   64 rows 19 / 27 / 32 / 52,     4096 rows 135 / 105 / 93 / 72
// Split pays where its tiles are no more than the CUs: 64 rows 17 us bf16 and
// 12 E4M3; with 8192 columns, k 4096 and 128 rows bf16 Split2 24, Small 31,
// Split 31.
// One step goes to grouped_thin_kernel; two to Short, three workgroups of which
// fit a CU and hide their fixed parts best.
// Groups are taken to hold rows / experts rows and to need 0.6 of a tile more.
// Where many rows belong to no group (the layer's whole routing table on an EP
// shard) that is too many: 128 pairs in 76 of 112 groups, 16 x 3584, 8.4 us as
// 128 rows and 14.7 as the first 128 of 1024.
// Where there is more than a round the last one of grouped rows, whose number
// is only estimated, is taken as 0.3.
enum Shape { kSmall, kMid, kShort, kLarge, kPair, kSplit, kSplit2, kThin, kFew };
Shape choose(GroupedMode mode, const GroupedArgs& a, int cus) {
  const bool wg = mode == kGWgrad, f8 = mode == kGFwd8 || mode == kGFwd8x;
  if ((mode == kGFwd || f8) && few_rows(a)) return kFew;
  const int q = f8 ? 128 : 64;
  const double mean = (double)a.rows / a.experts;
  const double steps = wg ? mean / 64 + 0.5 : (double)((a.K + q - 1) / q);
  if (steps <= 1 && (mode == kGFwd || mode == kGDgrad)) return kThin;
  if (steps <= 2 && !wg) return kShort;
  struct Cost { Shape shape; int bm, bn, per_cu; double one, all, one8, all8, fixed; };
  constexpr Cost kCosts[] = {
      {kSmall, 64, 64, 2, 0.45, 0.46, 0.57, 0.61, 3},   {kMid, 64, 128, 2, 0.53, 0.72, 0.85, 1.03, 3},
      {kLarge, 128, 128, 2, 0.80, 1.20, 1.00, 1.62, 4}, {kPair, 256, 256, 1, 1.35, 1.75, 1.60, 2.00, 8},
      {kSplit, 64, 32, 1, 0.14, 0.14, 0.15, 0.15, 8},   {kSplit2, 64, 64, 1, 0.20, 0.20, 0.27, 0.27, 9}};
  Shape best = kSmall;
  double least = 1e30;
  for (const Cost& c : kCosts) {
    if (c.shape == kPair && (mode == kGFwd8x || !narrow_ok(mode, a))) continue;
    if ((c.shape == kSplit || c.shape == kSplit2) && wg && a.pairs) continue;   // row indices are shared by waves
    double m;
    if (wg) m = (double)((a.M + c.bm - 1) / c.bm) * a.experts;
    else if (!a.offsets) m = (a.rows + c.bm - 1) / c.bm;
    else m = a.experts * std::max(1.0, mean / c.bm + 0.6);
    const double tiles = m * ((a.N + c.bn - 1) / c.bn), slots = (double)cus * c.per_cu;
    const double rounds = tiles <= slots ? 1 : (wg || !a.offsets ? std::ceil(tiles / slots) : tiles / slots + 0.3);
    const double step = tiles <= cus ? (f8 ? c.one8 : c.one) : (f8 ? c.all8 : c.all);
    const double cost = rounds * (steps * step + c.fixed);
    if (cost < least) {
      least = cost;
      best = c.shape;
    }
  }
  return best;
}

template <int MODE, bool IDX>
hipError_t launch_mode(GroupedArgs& a, int cus, hipStream_t s) {
  // bf16 results in 16-byte stores: 8192 rows x 3584 x 32 of dx 24 us, in 8-byte ones 31.  dw is mostly fp32, whose
  // four columns a lane are 16 bytes already.
  constexpr bool kP = MODE == kGDgrad;
  switch (choose((GroupedMode)MODE, a, cus)) {
    case kSmall: return launch_as<Cfg<64, 64, 2, 2, 3, 2, kP>, MODE, IDX>(a, cus, s);
    case kMid: return launch_as<Cfg<64, 128, 2, 2, 3, 2, kP>, MODE, IDX>(a, cus, s);
    case kShort:
      if constexpr (MODE != kGWgrad) return launch_as<Cfg<64, 128, 2, 2, 2, 3, kP>, MODE, IDX>(a, cus, s);
      break;
    case kLarge: return launch_as<Cfg<128, 128, 2, 2, 2, 2, kP>, MODE, IDX>(a, cus, s);
    case kPair:
      if constexpr (MODE != kGFwd8x) return launch_as<Cfg<256, 256, 2, 4, 2, 2, kP>, MODE, IDX, -1>(a, cus, s);
      break;
    case kSplit:
      if constexpr (!IDX) return launch_as<Cfg<64, 32, 1, 1, 3, 1, kP>, MODE, IDX, 4>(a, cus, s);
      break;
    case kSplit2:
      if constexpr (!IDX) return launch_as<Cfg<64, 64, 1, 1, 2, 1, kP>, MODE, IDX, 4>(a, cus, s);
      break;
    case kThin:
      if constexpr (MODE == kGFwd || MODE == kGDgrad) return launch_thin<Cfg<64, 128, 2, 2, 3, 4, true>, MODE>(a, cus, s);
      break;
    case kFew:
      if constexpr (MODE == kGFwd || MODE == kGFwd8 || MODE == kGFwd8x) return launch_grouped_few((GroupedMode)MODE, a, cus, s);
      break;
  }
  return hipErrorInvalidValue;
}

GroupedMode with_output(GroupedMode mode, const GroupedArgs& a) {
  return mode == kGFwd8 && a.out_f32 ? kGFwd8x : mode;
}
// Whether a weight gradient looks its rows up (IDX).
bool indexed(const GroupedArgs& a) { return a.pairs && (a.t_div.div || a.c_div.div); }

}  // namespace

const char* grouped_kernel_name(GroupedMode mode, const GroupedArgs& a, int cus) {
  const bool idx = mode == kGWgrad && indexed(a);
  switch (choose(with_output(mode, a), a, cus)) {
    case kSmall: return idx ? "grouped_kernel 64x64 indexed" : "grouped_kernel 64x64";
    case kMid: return idx ? "grouped_kernel 64x128 indexed" : "grouped_kernel 64x128";
    case kShort: return "grouped_kernel 64x128 short";
    case kLarge: return idx ? "grouped_kernel 128x128 indexed" : "grouped_kernel 128x128";
    case kPair: return idx ? "grouped_pair_kernel indexed" : "grouped_pair_kernel";
    case kSplit: return "grouped_split_kernel 64x32";
    case kSplit2: return "grouped_split_kernel 64x64";
    case kThin: return "grouped_thin_kernel";
    case kFew: return few_wide(a, cus) ? "grouped_few_kernel 32" : "grouped_few_kernel 16";
  }
  return nullptr;
}

hipError_t launch_grouped(GroupedMode mode, GroupedArgs& a, int cus, hipStream_t s) {
  mode = with_output(mode, a);
  switch (mode) {
    case kGFwd: return launch_mode<kGFwd, false>(a, cus, s);
    case kGFwd8: return launch_mode<kGFwd8, false>(a, cus, s);
    case kGFwd8x: return launch_mode<kGFwd8x, false>(a, cus, s);
    case kGDgrad: return launch_mode<kGDgrad, false>(a, cus, s);
    case kGWgrad:
      if (indexed(a)) return launch_mode<kGWgrad, true>(a, cus, s);
      return launch_mode<kGWgrad, false>(a, cus, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace situ
