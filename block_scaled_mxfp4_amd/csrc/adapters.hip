// Low-rank adapters of many requests beside a shared projection
// (situ_moe_adapters): out[r] = base[r] + c_i b_i (a_i x[r]), i the adapter of
// r's request.
//
// A batch of many rows takes two launches: t = c a_i x into the workspace, then out
// = base + b_i t.  They are bound by HBM: 8192 rows, 3584 to 7168, rank 32, take 18
// and 46 us, the second at 5.1 TB/s of base and out.  Few rows (decode) take one
// launch, a row a workgroup, bound by its memory latencies in turn: 64 rows of
// rank 16 in 8.3 us, 14.8 in two.
//
// The two work on tiles of up to 16 rows in the order of the batch, whatever
// requests they belong to, so that neither the host nor the grid needs to know
// the requests' lengths: a wave holds the requests that reach into its tile one
// a lane and takes them in turn.  Every request's product is kept by its own rows
// alone: what another request's adapter holds (infinities, NaN) does not reach
// them.
//
// Between the two, t is held as its output asks for.  For a bf16 out it is two bf16
// terms, high and low: they lose no more than 2^-16 of it, against the 2^-8 of out's
// own rounding.  For an fp32 out it is fp32, which the second product takes apart
// into three bf16 terms, exactly, so that a row has the accuracy that the one
// launch gives it.  With ranks up to 16 two terms fit in one instruction's 32
// columns.  Both take 4 bytes a value.  The third term costs the fp32 output 0 to
// 9 % (8192 rows, 3584 to 7168: rank 16 136 us either way, rank 32 137 us against
// 130 with two, rank 128 396 against 366).
#include <algorithm>

#include "routed.hpp"
#include "wave.hpp"

namespace situ {

namespace {

constexpr int kUpWaves = 4;

struct AdapterArgs {
  situ_moe_adapters_t p;
  uint16_t *high, *low;       // bf16 out: t as two bf16 terms, [rows][rank] each
  float* t;                   // fp32 out: t, [rows][rank]; else null
  int32_t tile;               // rows of a tile of the first product, 1 .. 16
  int32_t up_tile;            // of the second, 1 .. 16
  int32_t up_tiles;
  int32_t run;                // of them a wave takes in turn (one launch: columns of a workgroup)
  int32_t chunks;             // of 128 columns in n (one launch: of `run` columns)
};

// Sixty-four consecutive requests, one a lane.
struct Requests {
  int32_t first, begin, end, adapter;   // of lane i: request first + i
};
__device__ __forceinline__ void load_requests(const situ_moe_adapters_t& p, int first, int lane, Requests& q) {
  const int i = first + lane;
  q.first = first;
  q.begin = q.end = 0;
  q.adapter = -1;
  if (i < p.requests) {
    q.begin = p.offsets[i];
    q.end = p.offsets[i + 1];
    q.adapter = p.adapter[i];
    if (q.adapter >= p.adapters) q.adapter = -1;
  }
}
// The lanes whose requests have rows in [r0, r1), and whether the next 64 may have some too.
__device__ __forceinline__ uint64_t in_tile(const Requests& q, int r0, int r1) {
  return __ballot(max(q.begin, r0) < min(q.end, r1));
}
__device__ __forceinline__ bool reaches_on(const situ_moe_adapters_t& p, const Requests& q, int r1) {
  return q.first + 64 < p.requests && __builtin_amdgcn_readlane(q.end, 63) < r1;
}
// The first of 64 requests among which is the first that reaches into a tile from r0.
__device__ __forceinline__ int first_request(const situ_moe_adapters_t& p, int r0, int lane) {
  int lo = 0, size = p.requests;
  while (size > 64) {
    const int step = (size + 63) / 64;
    const int end = lo + (lane + 1) * step;          // of lane's share; shares that end by r0 are passed over
    const int n = __popcll(__ballot(end < p.requests && p.offsets[min(end, p.requests)] <= r0));
    lo += n * step;
    size = min(step, p.requests - lo);
  }
  return lo;
}
__device__ __forceinline__ int next_bit(uint64_t& m) {
  const int i = __ffsll((unsigned long long)m) - 1;
  m &= m - 1;
  return i;
}

// Sixteen bytes, zeros where there are none: the address is chosen and not the load branched around, since behind
// branches the compiler cannot count the loads in flight and waits for all of them.
__device__ const uint4 kZeros[1] = {};
typedef const i32x4 __attribute__((address_space(1)))* Sixteen;
__device__ __forceinline__ Sixteen sixteen(const void* p, bool in) {
  const Sixteen at = (Sixteen)p, zeros = (Sixteen)kZeros;
  return in ? at : zeros;
}
__device__ __forceinline__ uint4 load16(const void* p, bool in) { return __builtin_bit_cast(uint4, *sixteen(p, in)); }
// Read once: past the caches, which a and t then stay in (8192 rows, the first product: 24 us, 21 so).
__device__ __forceinline__ uint4 load16_once(const void* p, bool in) {
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load(sixteen(p, in)));
}
__device__ __forceinline__ f32x4 mfma(const uint4& a, const uint4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ void unpack8(const uint4& v, float f[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_to_f32(w[i] & 0xffffu);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float f[8]) {
  const bf16x8 b = {(__bf16)f[0], (__bf16)f[1], (__bf16)f[2], (__bf16)f[3],
                    (__bf16)f[4], (__bf16)f[5], (__bf16)f[6], (__bf16)f[7]};   // nearest even
  return __builtin_bit_cast(uint4, b);
}

// Four ranks of t as two bf16 terms.  A value that is not finite has no second; a finite one past bf16's largest has
// that as its first.
__device__ __forceinline__ void two_terms(const f32x4& t, uint2& high, uint2& low) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  bf16x4 h, l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = (__bf16)t[i];
    if (fabsf((float)h[i]) == __builtin_inff() && fabsf(t[i]) < __builtin_inff())
      h[i] = (__bf16)__builtin_copysignf(0x1.fep127f, t[i]);
    const float d = t[i] - (float)h[i];
    l[i] = (__bf16)(fabsf(d) < __builtin_inff() ? d : 0.0f);
  }
  high = __builtin_bit_cast(uint2, h);
  low = __builtin_bit_cast(uint2, l);
}
// Eight ranks of t as three bf16 terms: eight bits each of its 24, by cutting off, so that nothing is lost and a finite
// value has finite terms.  A value that is not finite has one term.
__device__ __forceinline__ void three_terms(const uint4& lo, const uint4& hi, uint4 term[3]) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t cut[3][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float left = __uint_as_float(w[i]);
#pragma unroll
    for (int o = 0; o < 3; ++o) {
      cut[o][i] = __float_as_uint(left) & 0xffff0000u;
      left -= __uint_as_float(cut[o][i]);
      left = fabsf(left) < __builtin_inff() ? left : 0.0f;
    }
  }
#pragma unroll
  for (int o = 0; o < 3; ++o)
    term[o] = make_uint4(cut[o][0] >> 16 | cut[o][1], cut[o][2] >> 16 | cut[o][3], cut[o][4] >> 16 | cut[o][5],
                         cut[o][6] >> 16 | cut[o][7]);
}

// t.  A workgroup takes a tile of rows, its waves every W-th unit of 64 of k.  A unit of x and a is requested by
// whole lines, eight lanes of 16 bytes a row (rows of 64 bytes, as the matrix instruction holds them, go through the
// address unit at half the rate: 8192 x 3584 of rank 32 in 36 us), put into the wave's own LDS and read back as
// operands: lane l ranks 16 i + l % 16 of a (rows of the instruction) and token l % 16 of x (columns), eight of k, so
// that it ends with four consecutive ranks of a token.  Piece c of row r lies in place c ^ (r % 8).  The next unit is
// under way while one is multiplied; waves in number hide the rest (17.8 us; two and three units ahead, with the
// registers of fewer waves, 19 and 21; tiles of 32 rows the same).  RT: tiles of 16 ranks.
template <int RT, int W>
__global__ __launch_bounds__(64 * W) void adapters_down_kernel(AdapterArgs a) {
  constexpr int kParts = 2 * (RT + 1);                // of eight rows in a unit
  __shared__ uint4 lds[W][kParts * 64];
  const situ_moe_adapters_t& p = a.p;
  const int lane = lane_id(), wave = wave_id(), col = lane & 15, group = lane >> 4;
  const int line = lane >> 3, piece = lane & 7;
  const int r0 = blockIdx.x * a.tile, r1 = min(r0 + a.tile, p.rows);
  const int units = (p.k + 63) / 64;
  uint4* mine = lds[wave];
  const uint16_t* x[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) x[j] = p.x + (int64_t)min(r0 + 8 * j + line, r1 - 1) * p.x_stride + 8 * piece;
  Requests q;
  for (int first = first_request(p, r0, lane);; first += 64) {
    load_requests(p, first, lane, q);
    uint64_t some = in_tile(q, r0, r1);
    while (some) {
      const int at = next_bit(some);
      const int i = __builtin_amdgcn_readlane(q.adapter, at);
      if (i < 0) continue;
      const int lo = max(__builtin_amdgcn_readlane(q.begin, at), r0);
      const int hi = min(__builtin_amdgcn_readlane(q.end, at), r1);
      const float c = p.scales ? p.scales[i] : 1.0f;
      const int rank = p.ranks ? min(max(p.ranks[i], 0), p.rank) : p.rank;
      const uint16_t* w[2 * RT];
#pragma unroll
      for (int j = 0; j < 2 * RT; ++j)
        w[j] = p.a + ((int64_t)i * p.rank + min(8 * j + line, p.rank - 1)) * p.k + 8 * piece;
      f32x4 acc[RT];
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[j] = f32x4{0, 0, 0, 0};
      uint4 v[kParts];
      auto request = [&](int u) {                     // of units past the last: zeros
        const bool in = u < units && u * 64 + 8 * piece < p.k;
#pragma unroll
        for (int j = 0; j < 2; ++j) v[j] = load16(x[j] + u * 64, in);
#pragma unroll
        for (int j = 0; j < 2 * RT; ++j) v[2 + j] = load16(w[j] + u * 64, in);
      };
      request(wave);
      for (int u = wave; u < units; u += W) {
#pragma unroll
        for (int j = 0; j < kParts; ++j) mine[64 * j + 8 * line + (piece ^ line)] = v[j];
        wave_lds();
        request(u + W);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = (4 * h + group) ^ (col & 7);
          const uint4 xt = mine[8 * col + c];
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[j] = mfma(mine[8 * (16 * (1 + j) + col) + c], xt, acc[j]);
        }
        wave_lds();
      }
      // the waves' sums: each wave adds up every W-th tile of 16 ranks
#pragma unroll
      for (int j = 0; j < RT; ++j) mine[64 * j + lane] = __builtin_bit_cast(uint4, acc[j]);
      __syncthreads();
      for (int j = wave; j < RT; j += W) {
        f32x4 t = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < W; ++e) t += __builtin_bit_cast(f32x4, lds[e][64 * j + lane]);
        const int r = 16 * j + 4 * group, row = r0 + col;
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = r + e < rank ? t[e] * c : 0.0f;
        if (row < lo || row >= hi || r >= p.rank) continue;
        if (a.t) {
          *reinterpret_cast<f32x4*>(a.t + (int64_t)row * p.rank + r) = t;
        } else {
          uint2 high, low;
          two_terms(t, high, low);
          *reinterpret_cast<uint2*>(a.high + (int64_t)row * p.rank + r) = high;
          *reinterpret_cast<uint2*>(a.low + (int64_t)row * p.rank + r) = low;
        }
      }
      __syncthreads();                                // before the next request's units take their place
    }
    if (!reaches_on(p, q, r1)) break;
  }
}

// out.  Tokens are the rows of the instruction and columns of out its columns: lane l holds token l % 16, eight ranks
// from 8 (l / 16), and of instruction s column 8 (l % 16) + s, so that it ends with eight consecutive columns of the
// four tokens 4 (l / 16) ..: 16 bytes of bf16, 256 consecutive ones a token.  A wave takes 128 columns of a run of
// tiles and keeps its columns of b while the adapter stays the same (KEEP: up to 64 ranks).
// KS: steps of 32 ranks; 0: at most 16 ranks, the second term beside the first in one instruction.
template <int KS, bool F32>
__global__ __launch_bounds__(64 * kUpWaves) void adapters_up_kernel(AdapterArgs a, int64_t items) {
  constexpr int S = KS ? KS : 1, NB = F32 ? 2 : 1;
  constexpr int kTerms = F32 ? 3 : 2, kMany = KS ? kTerms : kTerms - 1;    // instructions a step of ranks and column
  constexpr bool KEEP = S <= 2;
  const situ_moe_adapters_t& p = a.p;
  const int lane = lane_id(), col = lane & 15, group = lane >> 4;
  const int64_t item = (int64_t)blockIdx.x * kUpWaves + wave_id();
  if (item >= items) return;
  const int run = (int)((uint32_t)item / (uint32_t)a.chunks), chunk = (int)((uint32_t)item - (uint32_t)run * a.chunks);
  const int c = chunk * 128 + 8 * col;               // the lane's eight columns
  const bool in = c < p.n;
  const int r_at = KS ? 8 * group : 8 * (group & 1); // its ranks, of each 32
  auto load_b = [&](const uint16_t* w, int rank, int s, int ks) {
    const int r = 32 * ks + r_at;
    uint4 f = load16(w + s * p.rank + 32 * ks, in && r < rank);
    if (r + 8 > rank) {                              // columns past the adapter's own rank
      uint32_t g[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (r + 2 * e >= rank) g[e] = 0;
        else if (r + 2 * e + 1 >= rank) g[e] &= 0xffffu;
      }
      f = make_uint4(g[0], g[1], g[2], g[3]);
    }
    return f;
  };
  const int tile1 = min((run + 1) * a.run, a.up_tiles);
  // what a tile needs of base and of t, requested while the one before is computed
  struct Tile { uint4 base[4][NB], t[F32 || KS ? 2 : 1][S]; };   // t: the two terms, or ranks 0 .. 3 and 4 .. 7 in fp32
  const char* base_at = static_cast<const char*>(p.base);
  auto request = [&](Tile& f, int tile) {
    const int r0 = tile * a.up_tile, r1 = tile < tile1 ? min(r0 + a.up_tile, p.rows) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r0 + 4 * group + i;
#pragma unroll
      for (int h = 0; h < NB; ++h)
        f.base[i][h] = load16_once(base_at + ((int64_t)row * p.base_stride + c) * (F32 ? 4 : 2) + 16 * h,
                                   p.base && in && row < r1);
    }
    // of token l % 16: rows of requests without an adapter hold anything, and are not used
    const int64_t t = (int64_t)(r0 + col) * p.rank + r_at;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const bool on = 32 * s + r_at < p.rank && r0 + col < r1;
      if constexpr (F32) {
        f.t[0][s] = load16(a.t + t + 32 * s, on);
        f.t[F32 || KS ? 1 : 0][s] = load16(a.t + t + 32 * s + 4, on);
      } else if constexpr (KS == 0) {
        f.t[0][s] = load16((group < 2 ? a.high : a.low) + t, on);
      } else {
        f.t[0][s] = load16(a.high + t + 32 * s, on);
        f.t[KS ? 1 : 0][s] = load16(a.low + t + 32 * s, on);
      }
    }
  };
  Tile now;
  request(now, run * a.run);
  Requests q;
  load_requests(p, first_request(p, run * a.run * a.up_tile, lane), lane, q);
  int held = -1;                                     // the adapter whose b is kept
  uint4 b[KEEP ? S : 1][8];
  for (int tile = run * a.run; tile < tile1; ++tile) {
    const int r0 = tile * a.up_tile, r1 = min(r0 + a.up_tile, p.rows);
    const int mine = r0 + 4 * group;                 // the first of the lane's four rows of out
    const Tile f = now;
    request(now, tile + 1);
    uint4 op[kMany][S];                              // the terms as operands
#pragma unroll
    for (int ks = 0; ks < S; ++ks) {
      if constexpr (F32) {
        uint4 term[3];
        three_terms(f.t[0][ks], f.t[F32 || KS ? 1 : 0][ks], term);
        if constexpr (KS == 0) {
          op[0][ks] = group < 2 ? term[0] : term[1];
          op[kMany - 1][ks] = group < 2 ? term[2] : make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
          for (int o = 0; o < kMany; ++o) op[o][ks] = term[o];
        }
      } else {
#pragma unroll
        for (int o = 0; o < kMany; ++o) op[o][ks] = f.t[o][ks];
      }
    }
    f32x4 sum[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) sum[s] = f32x4{0, 0, 0, 0};
    uint32_t of_request = 0;                         // bit i: row mine + i has a request
    for (;;) {
      uint64_t some = in_tile(q, r0, r1);
      while (some) {
        const int at = next_bit(some);
        const int i = __builtin_amdgcn_readlane(q.adapter, at);
        const int lo = __builtin_amdgcn_readlane(q.begin, at), hi = min(__builtin_amdgcn_readlane(q.end, at), r1);
        uint32_t own = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) own |= (mine + e >= lo && mine + e < hi ? 1u : 0u) << e;
        of_request |= own;
        if (i < 0) continue;
        const int rank = p.ranks ? min(max(p.ranks[i], 0), p.rank) : p.rank;
        const uint16_t* w = p.b + ((int64_t)i * p.n + c) * p.rank + r_at;
        if (KEEP && i != held) {
          held = i;
#pragma unroll
          for (int s = 0; s < 8; ++s)
#pragma unroll
            for (int ks = 0; ks < S; ++ks) b[KEEP ? ks : 0][s] = load_b(w, rank, s, ks);
        }
        const bool all = lo <= r0 && hi >= r1;       // the tile is this request's alone
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          f32x4 v = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int ks = 0; ks < S; ++ks) {
            const uint4 g = KEEP ? b[KEEP ? ks : 0][s] : load_b(w, rank, s, ks);
#pragma unroll
            for (int o = 0; o < kMany; ++o) v = mfma(op[o][ks], g, v);
          }
          if (all) {
            sum[s] = v;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[s][e] = own >> e & 1 ? v[e] : sum[s][e];
          }
        }
      }
      if (!reaches_on(p, q, r1)) break;
      load_requests(p, q.first + 64, lane, q);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!in || !(of_request >> i & 1)) continue;
      float o[8];
      if constexpr (F32) {
        const uint32_t u[8] = {f.base[i][0].x, f.base[i][0].y, f.base[i][0].z, f.base[i][0].w,
                               f.base[i][NB - 1].x, f.base[i][NB - 1].y, f.base[i][NB - 1].z, f.base[i][NB - 1].w};
#pragma unroll
        for (int s = 0; s < 8; ++s) o[s] = __uint_as_float(u[s]) + sum[s][i];
        float* to = static_cast<float*>(p.out) + (int64_t)(mine + i) * p.out_stride + c;
        *reinterpret_cast<f32x4*>(to) = f32x4{o[0], o[1], o[2], o[3]};
        *reinterpret_cast<f32x4*>(to + 4) = f32x4{o[4], o[5], o[6], o[7]};
      } else {
        unpack8(f.base[i][0], o);
#pragma unroll
        for (int s = 0; s < 8; ++s) o[s] += sum[s][i];
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (int64_t)(mine + i) * p.out_stride + c) = pack8(o);
      }
    }
  }
}

// One row, as decode's requests have: both products in one launch.  A workgroup takes a row and a share of out's
// columns, and computes t for itself: a wave takes every eighth rank, its lanes eight of k at a time.  The row's
// workgroups lie on one die (workgroups go round the eight dies), so that a is read into one cache.  Of b, as many
// lanes as a row of it has pieces of eight ranks (the next power of two) share a column; its first pieces and base are
// requested before t is known.
constexpr int kRowWaves = 8, kRowPieces = 2, kRowCols = kRowPieces * 64 * kRowWaves * 8, kRowAhead = 8;
template <bool F32>
__global__ __launch_bounds__(64 * kRowWaves) void adapters_row_kernel(AdapterArgs a, int log_pieces) {
  __shared__ float ts[256], sums[kRowCols];
  const situ_moe_adapters_t& p = a.p;
  const int lane = lane_id(), wave = wave_id();
  const int slot = blockIdx.x / 8, row = slot / a.chunks * 8 + blockIdx.x % 8, chunk = slot % a.chunks;
  if (row >= p.rows) return;
  const int c0 = chunk * a.run, c1 = min(c0 + a.run, p.n);       // run: columns of a workgroup
  // base: eight columns a thread and piece
  constexpr int NB = F32 ? 2 : 1;
  const char* base_at = static_cast<const char*>(p.base);
  uint4 base[kRowPieces][NB];
#pragma unroll
  for (int o = 0; o < kRowPieces; ++o) {
    const int c = c0 + 8 * ((int)threadIdx.x + 64 * kRowWaves * o);
#pragma unroll
    for (int h = 0; h < NB; ++h)
      base[o][h] = load16(base_at + ((int64_t)row * p.base_stride + c) * (F32 ? 4 : 2) + 16 * h, p.base && c < c1);
  }
  // x: eight of k a lane and piece
  const uint16_t* xr = p.x + (int64_t)row * p.x_stride;
  uint4 x[kRowAhead];
#pragma unroll
  for (int o = 0; o < kRowAhead; ++o) x[o] = load16(xr + 8 * (lane + kWave * o), 8 * (lane + kWave * o) < p.k);
  Requests q;
  uint64_t some = 0;
  for (int first = first_request(p, row, lane);; first += 64) {
    load_requests(p, first, lane, q);
    some = in_tile(q, row, row + 1);
    if (some || !reaches_on(p, q, row + 1)) break;
  }
  if (!some) return;                                 // of no request
  const int i = __builtin_amdgcn_readlane(q.adapter, next_bit(some));
  const bool adapted = i >= 0;
  const int rank = !adapted ? 0 : p.ranks ? min(max(p.ranks[i], 0), p.rank) : p.rank;
  if (rank > 0) {
    const int pieces = 1 << log_pieces, mine = lane & (pieces - 1), cols = kWave >> log_pieces;
    const uint16_t* b = p.b + (int64_t)i * p.n * p.rank + 8 * mine;
    const int step = kRowWaves * cols, cw = c0 + wave * cols + (lane >> log_pieces);
    uint4 ahead[kRowAhead];
#pragma unroll
    for (int o = 0; o < kRowAhead; ++o)
      ahead[o] = load16(b + (int64_t)(cw + o * step) * p.rank, 8 * mine < rank && cw + o * step < c1);
    __builtin_amdgcn_sched_barrier(0);
    const float scale = p.scales ? p.scales[i] : 1.0f;
    const uint16_t* w = p.a + (int64_t)i * p.rank * p.k;
    for (int r = wave; r < p.rank; r += 2 * kRowWaves) {
      const bool two = r + kRowWaves < rank;
      const uint16_t* w0 = w + (int64_t)r * p.k;
      const uint16_t* w1 = w0 + (two ? (int64_t)kRowWaves * p.k : 0);
      float s0 = 0.0f, s1 = 0.0f;
      for (int k0 = 0; k0 < p.k; k0 += 8 * kWave * kRowAhead) {
        uint4 v0[kRowAhead], v1[kRowAhead];
#pragma unroll
        for (int o = 0; o < kRowAhead; ++o) {
          const int k = k0 + 8 * (lane + kWave * o);
          v0[o] = load16(w0 + k, k < p.k);
          v1[o] = load16(w1 + k, k < p.k);
        }
#pragma unroll
        for (int o = 0; o < kRowAhead; ++o) {
          const int k = k0 + 8 * (lane + kWave * o);
          float fx[8], f0[8], f1[8];
          unpack8(k0 == 0 ? x[o] : load16(xr + k, k < p.k), fx);
          unpack8(v0[o], f0);
          unpack8(v1[o], f1);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s0 = fmaf(fx[e], f0[e], s0);
            s1 = fmaf(fx[e], f1[e], s1);
          }
        }
      }
      s0 = wave_sum(s0);
      s1 = wave_sum(s1);
      if (lane == 0) {
        ts[r] = r < rank ? s0 * scale : 0.0f;
        if (r + kRowWaves < p.rank) ts[r + kRowWaves] = two ? s1 * scale : 0.0f;
      }
    }
    __syncthreads();
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = 8 * mine + e < rank ? ts[8 * mine + e] : 0.0f;
    auto finish = [&](const uint4& v, int c) {
      float f[8], s = 0.0f;
      unpack8(v, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = 8 * mine + e < rank ? fmaf(f[e], t[e], s) : s;
      for (int m = 1; m < pieces; m *= 2) s += __shfl_xor(s, m, kWave);
      if (mine == 0 && c < c1) sums[c - c0] = s;
    };
#pragma unroll
    for (int o = 0; o < kRowAhead; ++o)
      if (c0 + wave * cols + o * step < c1) finish(ahead[o], cw + o * step);
    for (int c = cw + kRowAhead * step; c - (lane >> log_pieces) < c1; c += step)
      finish(load16(b + (int64_t)c * p.rank, 8 * mine < rank && c < c1), c);
    __syncthreads();
  }
#pragma unroll
  for (int o = 0; o < kRowPieces; ++o) {
    const int at = 8 * ((int)threadIdx.x + 64 * kRowWaves * o), c = c0 + at;
    if (c >= c1) continue;
    float f[8];
    if constexpr (F32) {
      const uint4 u = base[o][0], v = base[o][NB - 1];
      const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(w[e]);
    } else {
      unpack8(base[o][0], f);
    }
    if (rank > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += sums[at + e];
    }
    if constexpr (F32) {
      float* to = static_cast<float*>(p.out) + (int64_t)row * p.out_stride + c;
      *reinterpret_cast<f32x4*>(to) = f32x4{f[0], f[1], f[2], f[3]};
      *reinterpret_cast<f32x4*>(to + 4) = f32x4{f[4], f[5], f[6], f[7]};
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (int64_t)row * p.out_stride + c) = pack8(f);
    }
  }
}

// Tiles of the two launches: as many of the first product's as there are CUs, where there are rows for them.
int up_tile_rows(int32_t rows) { return rows <= 64 ? 1 : rows <= 256 ? 4 : 16; }
int down_tile_rows(int32_t rows) {
  int tile = 1;
  while (tile < 16 && rows > 256 * tile) tile *= 2;
  return tile;
}
// The one launch reads both matrices of its adapter for every row; two launches read them once for the rows of a request
// in a tile.  Rank 16, 3584 to 7168, requests of one row: 64 rows 8.7 us against 14.8, 256 rows 20 against 27; rank 32:
// 64 rows 14 against 17, 128 rows 22 against 21.  Requests of 32 rows, rank 16: 64 rows 8.8 against 12.1, 128 rows 12.4
// against 12.6, 256 rows 20 against 15.  Larger ranks, requests of one row: 16 rows 11 against 15 at rank 64, 22 against
// 25 at 128, 42 against 56 at 256; 32 rows 17 against 18, 31 against 28, 62 against 74; 64 rows 23 against 23, 46 against
// 35, 96 against 107.  One request of 64 rows: 20 against 18, 39 against 34, 92 against 78.  So 64 rows of rank 128 are
// a quarter slower than they could be.
bool row_by_row(const situ_moe_adapters_t& p) {
  if (p.rank > 16) return p.rows <= 64;
  return p.rows <= 128 || (p.rows <= 512 && p.rows <= 2 * (int64_t)p.requests);
}

template <bool F32>
void up_go(const AdapterArgs& a, int64_t items, hipStream_t s) {
  const dim3 grid((unsigned)((items + kUpWaves - 1) / kUpWaves)), threads(64 * kUpWaves);
  const int r = a.p.rank;
  if (r <= 16) hipLaunchKernelGGL((adapters_up_kernel<0, F32>), grid, threads, 0, s, a, items);
  else if (r <= 32) hipLaunchKernelGGL((adapters_up_kernel<1, F32>), grid, threads, 0, s, a, items);
  else if (r <= 64) hipLaunchKernelGGL((adapters_up_kernel<2, F32>), grid, threads, 0, s, a, items);
  else if (r <= 128) hipLaunchKernelGGL((adapters_up_kernel<4, F32>), grid, threads, 0, s, a, items);
  else hipLaunchKernelGGL((adapters_up_kernel<8, F32>), grid, threads, 0, s, a, items);
}

}  // namespace

uint64_t adapters_workspace_bytes(const situ_moe_adapters_t& p) {
  return row_by_row(p) ? 0 : 4ull * (uint64_t)p.rows * (uint64_t)p.rank;
}

hipError_t launch_adapters(const situ_moe_adapters_t& p, hipStream_t s) {
  AdapterArgs a{};
  a.p = p;
  const int r = p.rank;
  if (row_by_row(p)) {
    // workgroups of a row: 256 in all, each 256 to 8192 columns
    const int eights = (p.rows + 7) / 8;
    const int most = (p.n + 255) / 256, least = (p.n + kRowCols - 1) / kRowCols;
    a.chunks = std::max({1, least, std::min(most, 32 / eights)});
    a.run = ((p.n + a.chunks - 1) / a.chunks + 7) / 8 * 8;
    a.chunks = (p.n + a.run - 1) / a.run;
    int log_pieces = 0;
    while (8 << log_pieces < r) ++log_pieces;
    const dim3 grid((unsigned)(eights * 8 * a.chunks)), threads(64 * kRowWaves);
    if (p.out_dtype == SITU_OUT_F32) hipLaunchKernelGGL(adapters_row_kernel<true>, grid, threads, 0, s, a, log_pieces);
    else hipLaunchKernelGGL(adapters_row_kernel<false>, grid, threads, 0, s, a, log_pieces);
    return hipGetLastError();
  }
  if (p.out_dtype == SITU_OUT_F32) {
    a.t = static_cast<float*>(p.workspace);
  } else {
    a.high = static_cast<uint16_t*>(p.workspace);
    a.low = a.high + (int64_t)p.rows * r;
  }
  a.up_tile = up_tile_rows(p.rows);
  a.tile = down_tile_rows(p.rows);
  const dim3 grid((unsigned)((p.rows + a.tile - 1) / a.tile));
  if (r <= 16) hipLaunchKernelGGL((adapters_down_kernel<1, 8>), grid, dim3(512), 0, s, a);
  else if (r <= 32) hipLaunchKernelGGL((adapters_down_kernel<2, 8>), grid, dim3(512), 0, s, a);
  else if (r <= 64) hipLaunchKernelGGL((adapters_down_kernel<4, 8>), grid, dim3(512), 0, s, a);
  else if (r <= 128) hipLaunchKernelGGL((adapters_down_kernel<8, 8>), grid, dim3(512), 0, s, a);
  else hipLaunchKernelGGL((adapters_down_kernel<16, 4>), grid, dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.up_tiles = (p.rows + a.up_tile - 1) / a.up_tile;
  a.chunks = (p.n + 127) / 128;
  // tiles of a wave: as many as leave three waves for each of the chip's 1024 SIMDs
  constexpr int64_t kUpItems = 256 * 4 * 3;
  a.run = (int)std::min<int64_t>(std::max<int64_t>(1, ((int64_t)a.up_tiles * a.chunks + kUpItems - 1) / kUpItems), a.up_tiles);
  const int64_t items = (int64_t)((a.up_tiles + a.run - 1) / a.run) * a.chunks;
  if (p.out_dtype == SITU_OUT_F32) up_go<true>(a, items, s);
  else up_go<false>(a, items, s);
  return hipGetLastError();
}

}  // namespace situ
