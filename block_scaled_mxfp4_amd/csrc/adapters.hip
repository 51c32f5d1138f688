// Low-rank adapters of many requests beside a shared projection
// (situ_moe_adapters): out[r] = base[r] + c_i b_i (a_i x[r]), i the adapter of
// r's request.
//
// Two launches: t = c a_i x in fp32 into the workspace, then out = base + b_i t.
// Prefill is bound by HBM (x read once, base and out once; the adapters come from
// L2), decode by the two launches and their memory latencies.
//
// Both work on tiles of up to 16 rows in the order of the batch, whatever
// requests they belong to, so that neither the host nor the grid needs to know
// the requests' lengths: a wave holds the requests that reach into its tile one
// a lane and takes them in turn.  Tokens lie on the column side of the matrix
// instruction, so that a lane ends with consecutive ranks, or columns of out, of
// one token.  Every request's product is kept by its own rows alone: what another
// request's adapter holds (infinities, NaN) does not reach them.
//
// The first product splits k over the waves of a workgroup and over workgroups
// (`parts`), whose sums the second one adds.  The second takes t as two bf16
// terms, high and low, so that no more than 2^-16 of it is lost; with ranks up to
// 16 both fit in one instruction's 32 columns.
#include <algorithm>

#include "routed.hpp"
#include "wave.hpp"

namespace situ {

namespace {

constexpr int kWaves = 4;

struct AdapterArgs {
  situ_moe_adapters_t p;
  float* t;                   // [parts][rows][rank]
  int32_t tile;               // rows of a tile, 1 .. 16
  int32_t tiles;
  int32_t parts;
  int32_t cols;               // the second product: columns of a wave, a multiple of 64
  int32_t chunks;             // of them in n
};

// The requests that reach into rows [r0, r1): a wave's lanes hold 64 consecutive ones.
struct Requests {
  int32_t first, lo, hi, adapter;   // of lane i: request first + i
  uint64_t some;                    // the lanes whose request has rows in the tile
  bool more;                        // the next 64 may reach into the tile too
};
__device__ __forceinline__ void requests_at(const situ_moe_adapters_t& p, int first, int r0, int r1, int lane, Requests& q) {
  q.first = first;
  q.lo = q.hi = 0;
  q.adapter = -1;
  const int i = first + lane;
  if (i < p.requests) {
    q.lo = max(p.offsets[i], r0);
    q.hi = min(p.offsets[i + 1], r1);
    q.adapter = p.adapter[i];
    if (q.adapter >= p.adapters) q.adapter = -1;
  }
  q.some = __ballot(q.lo < q.hi);
  q.more = first + 64 < p.requests && p.offsets[first + 64] < r1;
}
// The first request of 64 among which is the first that reaches into a tile from r0.
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

__device__ __forceinline__ uint4 load16(const uint16_t* p, bool in) {
  return in ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(const uint4& a, const uint4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// t.  Lane l holds ranks 16 i + l % 16 of a (rows of the instruction) and token l % 16 of x (columns), eight of k
// from 8 (l / 16); a step is 64 of k, whole lines.  RT: tiles of 16 ranks.
template <int RT>
__global__ __launch_bounds__(64 * kWaves) void adapters_down_kernel(AdapterArgs a) {
  __shared__ f32x4 part[kWaves - 1][RT][64];
  const situ_moe_adapters_t& p = a.p;
  const int lane = lane_id(), wave = threadIdx.x / kWave, col = lane & 15, group = lane >> 4;
  const int tile = blockIdx.x % a.tiles, piece = blockIdx.x / a.tiles;
  const int r0 = tile * a.tile, r1 = min(r0 + a.tile, p.rows);
  const int units = (p.k + 63) / 64;
  const int u0 = (int)((int64_t)units * piece / a.parts), u1 = (int)((int64_t)units * (piece + 1) / a.parts);
  const int row = r0 + col;
  const uint16_t* x = p.x + (int64_t)min(row, r1 - 1) * p.x_stride;
  Requests q;
  q.more = true;
  for (int first = first_request(p, r0, lane); q.more; first += 64) {
    requests_at(p, first, r0, r1, lane, q);
    while (q.some) {
      const int at = next_bit(q.some);
      const int i = __builtin_amdgcn_readlane(q.adapter, at);
      if (i < 0) continue;
      const int lo = __builtin_amdgcn_readlane(q.lo, at), hi = __builtin_amdgcn_readlane(q.hi, at);
      const uint16_t* w = p.a + (int64_t)i * p.rank * p.k;
      f32x4 acc[RT];
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[j] = f32x4{0, 0, 0, 0};
      for (int u = u0 + wave; u < u1; u += kWaves) {
        const int k = u * 64 + 8 * group;
        const bool in0 = k < p.k, in1 = k + 32 < p.k;
        const uint4 x0 = load16(x + k, in0), x1 = load16(x + k + 32, in1);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          const uint16_t* v = w + (int64_t)min(16 * j + col, p.rank - 1) * p.k + k;
          acc[j] = mfma(load16(v, in0), x0, acc[j]);
          acc[j] = mfma(load16(v + 32, in1), x1, acc[j]);
        }
      }
      __syncthreads();                                // the last request's sums have been read
      if (wave > 0) {
#pragma unroll
        for (int j = 0; j < RT; ++j) part[wave - 1][j][lane] = acc[j];
      }
      __syncthreads();
      if (wave == 0) {
        const float c = p.scales ? p.scales[i] : 1.0f;
        const int rank = p.ranks ? min(max(p.ranks[i], 0), p.rank) : p.rank;
        float* out = a.t + ((int64_t)piece * p.rows + row) * p.rank;
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          f32x4 v = acc[j];
#pragma unroll
          for (int o = 0; o < kWaves - 1; ++o) v += part[o][j][lane];
          const int r = 16 * j + 4 * group;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = r + e < rank ? v[e] * c : 0.0f;
          if (row >= lo && row < hi && r < p.rank) *reinterpret_cast<f32x4*>(out + r) = v;
        }
      }
    }
  }
}

// Eight ranks of t as two bf16 terms.  A rounded value that is not finite has no second.
__device__ __forceinline__ void two_terms(const float t[8], uint4& high, uint4& low) {
  bf16x8 h, l;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = (__bf16)t[i];
    const float d = t[i] - (float)h[i];
    l[i] = (__bf16)(fabsf(d) < __builtin_inff() ? d : 0.0f);
  }
  high = __builtin_bit_cast(uint4, h);
  low = __builtin_bit_cast(uint4, l);
}

// out.  Lane l holds columns of out (rows of b, rows of the instruction) and
// token l % 16, eight ranks from 8 (l / 16).  Row m of instruction s is column 32
// (s / 2) + 8 (m / 4) + 4 (s % 2) + m % 4, so that a lane ends with eight
// consecutive columns of its token from each two: 16 bytes of bf16.
// KS: steps of 32 ranks; 0: at most 16 ranks, the low term beside the high one.
template <int KS, bool F32>
__global__ __launch_bounds__(64 * kWaves) void adapters_up_kernel(AdapterArgs a, int64_t items) {
  constexpr int S = KS ? KS : 1;
  const situ_moe_adapters_t& p = a.p;
  const int lane = lane_id(), col = lane & 15, group = lane >> 4;
  const int64_t item = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
  if (item >= items) return;
  const int tile = (int)((uint32_t)item / (uint32_t)a.chunks), chunk = (int)((uint32_t)item - (uint32_t)tile * a.chunks);
  const int r0 = tile * a.tile, r1 = min(r0 + a.tile, p.rows);
  const int row = r0 + col;
  const int first = first_request(p, r0, lane);
  Requests q;
  requests_at(p, first, r0, r1, lane, q);
  const bool whole = !q.more;                        // these 64 are all
  // t of the token: rows of requests without an adapter hold anything, and are not used
  uint4 high[S], low[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int r = KS ? 32 * s + 8 * group : 8 * (group & 1);
    float t[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (r < p.rank && row < r1) {
      const float* at = a.t + (int64_t)row * p.rank + r;
      for (int i = 0; i < a.parts; ++i, at += (int64_t)p.rows * p.rank) {
        const f32x4 u = *reinterpret_cast<const f32x4*>(at), v = *reinterpret_cast<const f32x4*>(at + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) { t[e] += u[e]; t[4 + e] += v[e]; }
      }
    }
    two_terms(t, high[s], low[s]);
    if (!KS && group >= 2) high[s] = low[s];
  }
  const int c1 = min((chunk + 1) * a.cols, p.n);
  for (int c0 = chunk * a.cols; c0 < c1; c0 += 64) {
    f32x4 sum[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) sum[s] = f32x4{0, 0, 0, 0};
    bool held = false;                               // the token has a request
    // base, while the adapters' products run
    uint4 b0[2], b1[2];
    const int64_t base = (int64_t)row * p.base_stride;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + 32 * h + 8 * group;
      b0[h] = b1[h] = make_uint4(0, 0, 0, 0);
      if (p.base && row < r1 && c < p.n) {
        if constexpr (F32) {
          const uint4* v = reinterpret_cast<const uint4*>(static_cast<const float*>(p.base) + base + c);
          b0[h] = v[0];
          b1[h] = v[1];
        } else {
          b0[h] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.base) + base + c);
        }
      }
    }
    int start = first;
    for (;;) {
      if (!whole) requests_at(p, start, r0, r1, lane, q);
      uint64_t some = q.some;
      while (some) {
        const int at = next_bit(some);
        const int i = __builtin_amdgcn_readlane(q.adapter, at);
        const bool mine = row >= __builtin_amdgcn_readlane(q.lo, at) && row < __builtin_amdgcn_readlane(q.hi, at);
        held = held || mine;
        if (i < 0) continue;
        const int rank = p.ranks ? min(max(p.ranks[i], 0), p.rank) : p.rank;
        const uint16_t* w = p.b + (int64_t)i * p.n * p.rank;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int c = c0 + 32 * (s / 2) + 8 * (col / 4) + 4 * (s % 2) + col % 4;
          f32x4 v = f32x4{0, 0, 0, 0};
#pragma unroll
          for (int ks = 0; ks < S; ++ks) {
            const int r = KS ? 32 * ks + 8 * group : 8 * (group & 1);
            uint4 f = load16(w + (int64_t)min(c, p.n - 1) * p.rank + r, r < rank);
            if (r + 8 > rank) {                      // columns past the adapter's own rank
              uint32_t g[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (r + 2 * e >= rank) g[e] = 0;
                else if (r + 2 * e + 1 >= rank) g[e] &= 0xffffu;
              }
              f = make_uint4(g[0], g[1], g[2], g[3]);
            }
            v = mfma(f, high[ks], v);
            if constexpr (KS != 0) v = mfma(f, low[ks], v);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[s][e] = mine ? v[e] : sum[s][e];
        }
      }
      if (whole || !q.more) break;
      start += 64;
    }
    if (held && row < r1) {
      const int64_t out = (int64_t)row * p.out_stride;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = c0 + 32 * h + 8 * group;
        if (c >= p.n) continue;
        const uint32_t u[4] = {b0[h].x, b0[h].y, b0[h].z, b0[h].w};
        float f[8];
        if constexpr (F32) {
          const uint32_t v[4] = {b1[h].x, b1[h].y, b1[h].z, b1[h].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[e] = __uint_as_float(u[e]) + sum[2 * h][e];
            f[4 + e] = __uint_as_float(v[e]) + sum[2 * h + 1][e];
          }
          float* o = static_cast<float*>(p.out) + out + c;
          *reinterpret_cast<f32x4*>(o) = f32x4{f[0], f[1], f[2], f[3]};
          *reinterpret_cast<f32x4*>(o + 4) = f32x4{f[4], f[5], f[6], f[7]};
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f[2 * e] = bf16_to_f32(u[e] & 0xffffu) + sum[2 * h][2 * e];
            f[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u) + sum[2 * h][2 * e + 1];
            f[4 + 2 * e] = bf16_to_f32(u[2 + e] & 0xffffu) + sum[2 * h + 1][2 * e];
            f[5 + 2 * e] = __uint_as_float(u[2 + e] & 0xffff0000u) + sum[2 * h + 1][2 * e + 1];
          }
          const bf16x8 b = {(__bf16)f[0], (__bf16)f[1], (__bf16)f[2], (__bf16)f[3],
                            (__bf16)f[4], (__bf16)f[5], (__bf16)f[6], (__bf16)f[7]};   // nearest even
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + out + c) = __builtin_bit_cast(uint4, b);
        }
      }
    }
  }
}

// Few rows: a row a tile, as decode's requests have one each; else whole tiles.
int tile_rows(int32_t rows) { return rows <= 64 ? 1 : rows <= 256 ? 4 : 16; }

template <bool F32>
void up_go(const AdapterArgs& a, int64_t items, hipStream_t s) {
  const dim3 grid((unsigned)((items + kWaves - 1) / kWaves)), threads(64 * kWaves);
  const int r = a.p.rank;
  if (r <= 16) hipLaunchKernelGGL((adapters_up_kernel<0, F32>), grid, threads, 0, s, a, items);
  else if (r <= 32) hipLaunchKernelGGL((adapters_up_kernel<1, F32>), grid, threads, 0, s, a, items);
  else if (r <= 64) hipLaunchKernelGGL((adapters_up_kernel<2, F32>), grid, threads, 0, s, a, items);
  else if (r <= 128) hipLaunchKernelGGL((adapters_up_kernel<4, F32>), grid, threads, 0, s, a, items);
  else hipLaunchKernelGGL((adapters_up_kernel<8, F32>), grid, threads, 0, s, a, items);
}

}  // namespace

int adapters_parts(int32_t rows, int32_t k, int32_t rank) {
  (void)rank;
  const int tiles = (rows + tile_rows(rows) - 1) / tile_rows(rows), units = (k + 63) / 64;
  return std::max(1, std::min({512 / std::max(tiles, 1), units / kWaves, 16}));
}

hipError_t launch_adapters(const situ_moe_adapters_t& p, hipStream_t s) {
  AdapterArgs a{};
  a.p = p;
  a.t = static_cast<float*>(p.workspace);
  a.tile = tile_rows(p.rows);
  a.tiles = (p.rows + a.tile - 1) / a.tile;
  a.parts = adapters_parts(p.rows, p.k, p.rank);
  const dim3 grid((unsigned)(a.tiles * a.parts)), threads(64 * kWaves);
  const int r = p.rank;
  if (r <= 16) hipLaunchKernelGGL(adapters_down_kernel<1>, grid, threads, 0, s, a);
  else if (r <= 32) hipLaunchKernelGGL(adapters_down_kernel<2>, grid, threads, 0, s, a);
  else if (r <= 64) hipLaunchKernelGGL(adapters_down_kernel<4>, grid, threads, 0, s, a);
  else if (r <= 128) hipLaunchKernelGGL(adapters_down_kernel<8>, grid, threads, 0, s, a);
  else hipLaunchKernelGGL(adapters_down_kernel<16>, grid, threads, 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // columns of a wave: as many as leave 8192 waves
  const int blocks = (p.n + 63) / 64;
  const int64_t per = std::max<int64_t>(1, (int64_t)a.tiles * blocks / 8192);
  a.cols = (int)std::min<int64_t>(per, blocks) * 64;
  a.chunks = (p.n + a.cols - 1) / a.cols;
  const int64_t items = (int64_t)a.tiles * a.chunks;
  if (p.out_dtype == SITU_OUT_F32) up_go<true>(a, items, s);
  else up_go<false>(a, items, s);
  return hipGetLastError();
}

}  // namespace situ
