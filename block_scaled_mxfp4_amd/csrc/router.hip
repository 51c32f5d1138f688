// The gate: expert ids and weights of each token, the balance loss, and the
// logits' gradient (situ_moe_router, situ_moe_router_backward).
//
// A wave takes a token at a time and holds its logits in registers, V J of them
// a lane: expert e = 64 V j + V lane + v.
//
// Choice without sorting.  Where top_k of the 64 lanes' largest logits reach a
// threshold, the top_k largest of all do; a bisection on the lanes' largest finds
// one that hardly more do (over their values, three or four steps, where one over the
// float's bits takes ten: 32768 x 64 16 us for 24).  What reaches it (some 1.3 top_k) is packed into LDS,
// one candidate a lane, and a candidate's place is the number of candidates before
// it.  Where more than 64 reach it, the wave takes the largest that is left top_k
// times instead.  That is slow, and it is not for rows of equals alone (32768 x 896
// of them, top 16: 262 us for 32): since the threshold goes by the lanes' largest,
// it meets some ordinary rows from a top_k of some 30 on, most from 40 on, and all
// where top_k passes the lanes that have experts (34 for 65 or 129 experts).
// Softmax with the loss, 32768 rows of 896: top 24 34 us, 32 137, 40 762, 64 1316;
// of 160: top 24 27 us, 32 142; of 65: top 16 22 us, 34 138.
//
// A selection by sigmoid + bias is compared in 64 bits, since the neighbours of
// 900 experts lie as near as fp32 rounds.  The threshold is taken on fp32 scores
// and lowered by more than twice their error, and only where two candidates are
// nearer than that are the candidates' scores computed again in 64 bits.
//
// Sigmoid scores are held divided by e^min(zmax, 0), which leaves their shares as
// they are: a row whose scores all underflow keeps its weights.
//
// Balance loss: a wave sums its tokens' shares in registers, the workgroup's
// waves add theirs in LDS, and each workgroup writes partial sums and counts; a
// second launch adds them in a fixed order, and its last workgroup (by a ticket)
// takes the loss.  One workgroup finishes by itself.
//
// Bound by instruction issue and HBM alike: 32768 x 896 fp32 with the loss takes 28
// us and 6 for the second launch, against 20 for the logits at HBM's rate and 22
// for the 350 vector instructions of a token.  Up to 128 experts the CU's one scalar
// unit binds as much as the vector units (32768 x 64: 16 us, some 160 instructions a
// token of each); there and with few registers, logits requested a token ahead gained
// nothing, and at 896 experts they cost (42 us, by the registers).
#include <algorithm>

#include "common.hpp"
#include "routed.hpp"
#include "wave.hpp"

namespace situ {

namespace {

constexpr float kL2e = 1.44269502162933349609375f;   // log2(e) rounded to fp32
constexpr int kRouterWaves = 8;                       // of a workgroup
constexpr int kRouterBlocks = 768;                    // workgroups at most where the loss is taken
// Of the gradient: 640 workgroups suit softmax scores of many experts.  us with 512, 640, 1024 and 1536: 16384 x 896 fp32
// 24.7, 23.5, 27.6, 31.8 and bf16 21.2, 21.3, 24.2, 26.7; 32768 x 256 fp32 19.0, 17.1, 16.3, 16.5.  Few experts would
// take more (32768 x 64 fp32 11.6, 11.5, 10.1, 9.7), sigmoids of many fewer (16384 x 896 fp32 28.5, 32.5, 31.7, 32.7).
constexpr int kBackWaves = 8, kBackBlocks = 640;
constexpr int kOneBlockTokens = 32;                   // up to here one workgroup finishes the loss by itself

// Keys ascend with the values; 0 is an expert that cannot be chosen (-inf, NaN).
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t u = __float_as_uint(z + 0.0f);       // -0 as +0
  const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return z > -__builtin_inff() ? k : 0u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// The same order with a place for -inf; NaN must not be given.
__device__ __forceinline__ uint32_t order_of(float z) {
  const uint32_t u = __float_as_uint(z);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float wave_most(float z) { return value_of(wave_max(order_of(z))); }
__device__ __forceinline__ uint64_t key_of(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x + 0.0);
  return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}

__device__ __forceinline__ float e_to(float x) { return __builtin_amdgcn_exp2f(x * kL2e); }

template <bool BF>
__device__ __forceinline__ float load_one(const void* logits, int64_t at) {
  return BF ? bf16_to_f32(static_cast<const uint16_t*>(logits)[at]) : static_cast<const float*>(logits)[at];
}

// The logits of a row, -inf past the last expert.
template <bool BF, int V, int J>
__device__ __forceinline__ void load_row(const void* logits, int64_t at, int lane, int experts, bool vec,
                                         float z[V * J]) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = 64 * V * j + V * lane;
    if constexpr (V == 2) {
      if (vec && e + 2 <= experts) {
        if constexpr (BF) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(logits) + at + e);
          z[2 * j] = bf16_to_f32(w & 0xffffu);
          z[2 * j + 1] = bf16_to_f32(w >> 16);
        } else {
          const f32x2 w = *reinterpret_cast<const f32x2*>(static_cast<const float*>(logits) + at + e);
          z[2 * j] = w[0];
          z[2 * j + 1] = w[1];
        }
        continue;
      }
    }
    if constexpr (V == 4) {
      if (vec && e + 4 <= experts) {
        if constexpr (BF) {
          const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(logits) + at + e);
          z[4 * j] = bf16_to_f32(w.x & 0xffffu); z[4 * j + 1] = bf16_to_f32(w.x >> 16);
          z[4 * j + 2] = bf16_to_f32(w.y & 0xffffu); z[4 * j + 3] = bf16_to_f32(w.y >> 16);
        } else {
          const f32x4 w = *reinterpret_cast<const f32x4*>(static_cast<const float*>(logits) + at + e);
#pragma unroll
          for (int v = 0; v < 4; ++v) z[4 * j + v] = w[v];
        }
        continue;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      z[V * j + v] = -__builtin_inff();
      if (e + v < experts)
        z[V * j + v] = load_one<BF>(logits, at + e + v);
    }
  }
}

// Scores of a row, up to a factor the whole row shares: e^(z - zmax), or
// sigmoid(z) e^-min(zmax, 0).  FAR: the difference is taken first.  Otherwise the
// rounding of shift log2 e is a factor of the row too, 2^-25 |shift| log2 e in the
// exponent: near 1 up to the 2^20 of is_far, but past fp32's range from 2^31 on.
template <bool SIG, bool FAR>
__device__ __forceinline__ float score(float z, float shift) {
  const float x = SIG ? fminf(z, 0.0f) : z;
  const float n = FAR ? e_to(x - shift) : __builtin_amdgcn_exp2f(fmaf(x, kL2e, -shift * kL2e));
  return SIG ? n * __builtin_amdgcn_rcpf(1.0f + e_to(-fabsf(z))) : n;
}
__device__ __forceinline__ bool is_far(float shift) { return fabsf(shift) > 0x1p20f; }
template <bool SIG>
__device__ __forceinline__ float score(float z, float shift) {
  return is_far(shift) ? score<SIG, true>(z, shift) : score<SIG, false>(z, shift);
}
template <bool SIG, int N>
__device__ __forceinline__ void scores(const float z[N], float shift, float s[N]) {
  if (is_far(shift)) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = score<SIG, true>(z[i], shift);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = score<SIG, false>(z[i], shift);
  }
}

struct RouterArgs {
  situ_moe_router_t p;
  int32_t vec;
  float* part_sum;            // [gridDim.x][experts], or null: one workgroup, or no balance loss
  int32_t* part_count;
  uint32_t* ticket;
};

__device__ __forceinline__ uint64_t readlane64(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// A wave's row of logits by expert, and the candidates' ids, then what they are ordered by.  The row's place takes the
// scores in 64 bits where more than 64 candidates ask for them.
template <int N, bool BIAS>
struct alignas(16) WaveRow {
  union {
    float z[64 * N];
    uint64_t wide[BIAS ? 64 * N : 1];
  };
  int32_t id[64];
};

// The logits of token t; -inf for a masked one and past the last.
template <bool BF, int V, int J>
__device__ __forceinline__ void load_token(const situ_moe_router_t& p, int64_t t, int lane, bool vec, float z[V * J]) {
  if (t < p.tokens && (!p.mask || p.mask[t])) {
    load_row<BF, V, J>(p.logits, t * p.logits_stride, lane, p.experts, vec, z);
  } else {
#pragma unroll
    for (int i = 0; i < V * J; ++i) z[i] = -__builtin_inff();
  }
}

template <bool BF, int V, int J, bool SIG, bool BIAS, bool BAL>
__global__ __launch_bounds__(64 * kRouterWaves, 4) void router_kernel(RouterArgs a) {
  constexpr int N = V * J;
  __shared__ WaveRow<N, BIAS> wave_rows[kRouterWaves];
  __shared__ float biases[BIAS ? 64 * N : 1];
  __shared__ float sums[BAL ? 64 * N : 1];
  __shared__ int32_t hits[BAL ? 64 * N : 1];
  const situ_moe_router_t& p = a.p;
  const int lane = lane_id(), wave = wave_id();
  const int experts = p.experts, top_k = p.top_k;
  WaveRow<N, BIAS>& cd = wave_rows[wave];
  float acc[BAL ? N : 1];
  if constexpr (BAL) {
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    for (int i = threadIdx.x; i < 64 * N; i += 64 * kRouterWaves) hits[i] = 0;
    if (a.ticket && blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;     // for the launch that follows
    __syncthreads();
  }
  float bias[BIAS ? N : 1];
  if constexpr (BIAS) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = 64 * V * (i / V) + V * lane + i % V;
      bias[i] = e < experts ? p.bias[e] : 0.0f;
      if (wave == 0) biases[e] = bias[i];
    }
    __syncthreads();
  }
  const int64_t step = (int64_t)gridDim.x * kRouterWaves;
  for (int64_t t = (int64_t)blockIdx.x * kRouterWaves + wave; t < p.tokens; t += step) {
    const int64_t row = t * top_k;
    float z[N], best = -__builtin_inff();
    load_token<BF, V, J>(p, t, lane, a.vec, z);
#pragma unroll
    for (int i = 0; i < N; ++i) best = fmaxf(best, z[i]);     // passes over NaN
    const float zmax = wave_most(best);
    const bool live = zmax > -__builtin_inff();      // the row has an expert to choose
    // what is compared: the logit, or the fp32 score with its bias
    float c[BIAS ? N : 1], sig[BIAS && BAL ? N : 1], top = zmax;
    if constexpr (BIAS) {
      best = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float sigmoid = __builtin_amdgcn_rcpf(1.0f + e_to(-z[i]));
        if constexpr (BAL) sig[i] = sigmoid;
        c[i] = z[i] > -__builtin_inff() ? sigmoid + bias[i] : -__builtin_inff();
        best = fmaxf(best, c[i]);
      }
      top = wave_most(best);
    }
    // a threshold that top_k of the lanes' largest reach (all lanes' that have an expert do reach the least of
    // them), or the lowest value of all: every expert that can be chosen
    float least = -3.40282347e38f;
    const bool some = best > -__builtin_inff();
    int reach = __popcll(__ballot(some));
    if (reach >= top_k) {
      const float low = -wave_most(some ? -best : -__builtin_inff());
      // by values first, a few steps where they are spread evenly; by keys where they span magnitudes or are infinite
      const float step = (top - low) * 0x1p-8f;
      int at = 0;
      uint32_t w = 128;
      while (reach > top_k + 4 && w) {
        const int mid = at + (int)w, n = __popcll(__ballot(best >= fmaf((float)mid, step, low)));
        w >>= 1;
        if (n >= top_k) {
          at = mid;
          reach = n;
        }
      }
      least = at ? fmaf((float)at, step, low) : low;
      if (reach > top_k + 4) {
        uint32_t lo = key_of(least), hi = key_of(top);
        while (reach > top_k + 4 && hi > lo + 1) {
          const uint32_t mid = lo + (hi - lo) / 2;
          const int n = __popcll(__ballot(best >= value_of(mid)));
          if (n >= top_k) {
            lo = mid;
            reach = n;
          } else {
            hi = mid;
          }
        }
        least = value_of(lo);
      }
      least = fmaxf(least, -3.40282347e38f);
      // the k-th largest fp32 score is `least` at the least; one is off by less than 2^-21 + 2^-23 of its magnitude
      if (BIAS && least < __builtin_inff()) least = fmaxf(least - 0x1p-19f * (1.0f + fabsf(least)), -3.40282347e38f);
    }
    // a lane's candidates as bits, the first the highest; then one of each lane at a time into LDS
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      mine = mine + mine + ((BIAS ? c[BIAS ? i : 0] : z[i]) >= least ? 1u : 0u);
      cd.z[64 * V * (i / V) + V * lane + i % V] = z[i];
    }
    int n = 0;
    for (uint64_t who = __ballot(mine != 0); who; who = __ballot(mine != 0)) {
      const int at = (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, n));
      const uint32_t i = N - 1 - (uint32_t)__builtin_ctz(mine | 0x80000000u);
      if (mine && at < 64) cd.id[at] = 64 * V * (i / V) + V * lane + i % V;
      mine &= mine - 1;
      n += __popcll(who);
    }
    wave_lds();
    int id = -1, place = lane;                       // a lane's expert and its place in the row
    float zc = 0.0f;
    if (n <= 64) {
      // a candidate's place is the number of those before it: four at a time from LDS, and up to 32 of them by both
      // halves of the wave, each against half of them
      const bool halves = n <= 32;
      const int sub = halves ? lane & 31 : lane, quads = ((halves ? (n + 1) / 2 : n) + 3) / 4;
      const int from = halves ? (lane >> 5) * 4 * quads : 0;
      if (sub < n) {
        id = cd.id[sub];
        zc = cd.z[id];
      }
      wave_lds();
      uint32_t before = 0;
      if constexpr (BIAS) {
        // fp32 tells all of them apart but for a token in some hundreds
        const float b = sub < n ? biases[id] : 0.0f;
        const float mine = __builtin_amdgcn_rcpf(1.0f + e_to(-zc)) + b, apart = 0x1p-19f * (1.0f + fabsf(mine));
        uint32_t near = 0;
        cd.id[lane] = __float_as_int(lane < n ? mine : __builtin_nanf(""));
        wave_lds();
        for (int o = 0; o < quads; ++o) {
          const f32x4 others = *reinterpret_cast<const f32x4*>(&cd.id[from + 4 * o]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            before += others[i] > mine;
            near += fabsf(others[i] - mine) <= apart || others[i] == mine;    // itself, and infinities, too
          }
        }
        if (halves) {
          before = halves_sum(near << 16 | before);
          near = before >> 16;
          before &= 0xffffu;
        }
        if (__ballot(lane < n && near > 1)) {
          const uint64_t key = key_of(1.0 / (1.0 + exp(-(double)zc)) + (double)b);
          before = 0;
          for (int o = 0; o < n; ++o) {
            const uint64_t other = readlane64(key, o);
            const int oid = __builtin_amdgcn_readlane(id, o);
            before += other > key || (other == key && oid < id);
          }
        }
      } else {
        // a bf16 logit leaves room for the id in 32 bits.  fp32 ones are hardly ever equal: equal ones leave places
        // double and others empty
        const uint32_t key = BF ? (key_of(zc) & 0xffff0000u) | (uint32_t)(0xffff - id) : key_of(zc);
        cd.id[lane] = (int32_t)(lane < n ? key : 0u);
        wave_lds();
        for (int o = 0; o < quads; ++o) {
          const uint4 others = *reinterpret_cast<const uint4*>(&cd.id[from + 4 * o]);
          before += others.x > key;
          before += others.y > key;
          before += others.z > key;
          before += others.w > key;
        }
        if (halves) before = halves_sum(before);
        if (!BF && wave_sum(lane < n ? (float)before : 0.0f) != 0.5f * (float)(n * (n - 1))) {
          const uint64_t key64 = (uint64_t)key_of(zc) << 32 | (uint32_t)~id;
          before = 0;
          for (int o = 0; o < n; ++o) before += readlane64(key64, o) > key64;
        }
      }
      if (lane < n) place = (int)before;
      else id = -1;                                  // of the other half
    } else {
      // the largest left, top_k times: the largest behind the last one in the order of (key, lowest id)
      if constexpr (BIAS) {
#pragma unroll
        for (int i = 0; i < N; ++i)
        {
          const bool can = c[BIAS ? i : 0] > -__builtin_inff();
          const double score64 = 1.0 / (1.0 + exp(-(double)z[i])) + (double)bias[BIAS ? i : 0];
          cd.wide[BIAS ? 64 * i + lane : 0] = can ? key_of(score64) : 0;
        }
      }
      wave_lds();
      uint64_t last = ~0ull;
      int last_id = -1;
      for (int o = 0; o < top_k; ++o) {
        uint64_t most = 0;
        int at = 0;
#pragma unroll 1
        for (int i = 0; i < N; ++i) {                // ascending ids: the first of equals stays
          const int e = 64 * V * (i / V) + V * lane + i % V;
          const uint64_t k = BIAS ? cd.wide[BIAS ? 64 * i + lane : 0] : (uint64_t)key_of(cd.z[e]);
          if (k > most && (k < last || (k == last && e > last_id))) { most = k; at = e; }
        }
        const uint32_t h = BIAS ? wave_max((uint32_t)(most >> 32)) : 0u;
        const uint32_t l = wave_max((uint32_t)(most >> 32) == h ? (uint32_t)most : 0u);
        last = (uint64_t)h << 32 | l;
        if (!last) break;
        last_id = (int)~wave_max(most == last ? ~(uint32_t)at : 0u);
        if (lane == o) id = last_id;
      }
      if (id >= 0) zc = load_one<BF>(p.logits, t * p.logits_stride + id);
    }
    const bool chosen = id >= 0 && place < top_k;
    // renormalized weights are shares of the chosen: their own largest is the one to be near
    float wshift = SIG ? 0.0f : zmax;
    if (SIG && p.renormalize) wshift = fminf(BIAS ? wave_most(chosen ? zc : -__builtin_inff()) : zmax, 0.0f);
    float w = chosen ? score<SIG>(zc, wshift) : 0.0f;
    float all = 0.0f;
    if (live && (BAL || (!SIG && !p.renormalize))) {
      float s[N];
      if (SIG && zmax > -4.0f) {                       // none is lost that is 2^-120 of the largest
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = BIAS && BAL ? sig[BIAS && BAL ? i : 0] : __builtin_amdgcn_rcpf(1.0f + e_to(-z[i]));
      } else {
        scores<SIG, N>(z, SIG ? fminf(zmax, 0.0f) : zmax, s);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) all += s[i];
      all = wave_sum(all);
      if constexpr (BAL) {
        const float r = __builtin_amdgcn_rcpf(all);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(s[i], r, acc[i]);
        if (chosen) atomicAdd(&hits[id], 1);
      }
    }
    const float total = p.renormalize ? wave_sum(w) : (SIG ? 1.0f : all);
    w = chosen ? p.scale * (w * __builtin_amdgcn_rcpf(total)) : 0.0f;
    // the lanes behind the candidates fill the places that none has
    if (chosen || (lane < top_k && (n > 64 || lane >= n))) {
      const int64_t at = row + place;
      p.ids[at] = id;
      const uint32_t b = __builtin_bit_cast(uint16_t, (__bf16)w);    // nearest even
      if (p.weights) {
        if (p.weights_dtype == SITU_OUT_F32)
          static_cast<float*>(p.weights)[at] = w;
        else
          static_cast<uint16_t*>(p.weights)[at] = (uint16_t)b;
      }
      if (p.packed) p.packed[at] = (int32_t)(b << 16 | ((uint32_t)id & 0xffffu));
    }
    wave_lds();
  }
  if constexpr (BAL) {
    // the waves' sums take their rows' place, and are added in a fixed order
#pragma unroll
    for (int i = 0; i < N; ++i) cd.z[64 * V * (i / V) + V * lane + i % V] = acc[i];
    __syncthreads();
    for (int e = threadIdx.x; e < 64 * N; e += 64 * kRouterWaves) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kRouterWaves; ++w) sum += wave_rows[w].z[e];
      sums[e] = sum;
    }
    __syncthreads();
    const bool alone = gridDim.x == 1;
    float* so = alone ? p.prob_sum : a.part_sum + (int64_t)blockIdx.x * experts;
    int32_t* co = alone ? p.counts : a.part_count + (int64_t)blockIdx.x * experts;
    for (int e = threadIdx.x; e < experts; e += 64 * kRouterWaves) { so[e] = sums[e]; co[e] = hits[e]; }
    if (alone && wave == 0) {
      float n = 0.0f, d = 0.0f;
      for (int e = lane; e < experts; e += 64) {
        n += (float)hits[e];
        d += (float)hits[e] * sums[e];
      }
      n = wave_sum(n);
      d = wave_sum(d);
      if (lane == 0) *p.loss = n > 0.0f ? (float)experts * (float)top_k * (d / n) / n : 0.0f;
    }
  }
}

// Sums of the workgroups' parts, 16 experts a workgroup, 64 parts at a time; the
// last one to finish takes the loss.  Results that one workgroup hands another are
// written and read past the caches of the dies, so that no fence has to write
// back a whole cache: waiting for the stores before the ticket is enough.
constexpr int kFinishWaves = 16, kFinishExperts = 16;
__global__ __launch_bounds__(64 * kFinishWaves) void router_finish_kernel(RouterArgs a, int parts) {
  __shared__ float s_sum[kFinishWaves][kFinishExperts];
  __shared__ int32_t s_count[kFinishWaves][kFinishExperts];
  __shared__ float s_c[kFinishWaves], s_d[kFinishWaves];
  __shared__ uint32_t place;
  const situ_moe_router_t& p = a.p;
  const int lane = lane_id(), wave = wave_id(), e = blockIdx.x * kFinishExperts + lane % kFinishExperts;
  constexpr int kAtOnce = 64 * kFinishWaves / kFinishExperts;
  float sum = 0.0f;
  int32_t count = 0;
  if (e < p.experts) {
#pragma unroll 4
    for (int i = threadIdx.x / kFinishExperts; i < parts; i += kAtOnce) {
      sum += a.part_sum[(int64_t)i * p.experts + e];
      count += a.part_count[(int64_t)i * p.experts + e];
    }
  }
#pragma unroll
  for (int m = kFinishExperts; m < kWave; m *= 2) {
    sum += __shfl_xor(sum, m, kWave);
    count += __shfl_xor(count, m, kWave);
  }
  if (lane < kFinishExperts) {
    s_sum[wave][lane] = sum;
    s_count[wave][lane] = count;
  }
  __syncthreads();
  if (wave == 0) {
    if (lane < kFinishExperts && e < p.experts) {
      for (int w = 1; w < kFinishWaves; ++w) { sum += s_sum[w][lane]; count += s_count[w][lane]; }
      __hip_atomic_store(&p.prob_sum[e], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(&p.counts[e], count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __builtin_amdgcn_s_waitcnt(0);                   // the stores have reached where the others look
    if (lane == 0) place = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (place + 1 != gridDim.x) return;
  float c = 0.0f, d = 0.0f;
  for (int i = threadIdx.x; i < p.experts; i += 64 * kFinishWaves) {
    const float n = (float)__hip_atomic_load(&p.counts[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    c += n;
    d += n * __hip_atomic_load(&p.prob_sum[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  s_c[wave] = wave_sum(c);
  s_d[wave] = wave_sum(d);
  __syncthreads();
  if (threadIdx.x == 0) {
    c = d = 0.0f;
    for (int w = 0; w < kFinishWaves; ++w) { c += s_c[w]; d += s_d[w]; }
    *p.loss = c > 0.0f ? (float)p.experts * (float)p.top_k * (d / c) / c : 0.0f;
  }
}

// The gradient, bound by HBM (16384 x 896 fp32: 24 us, 4.9 TB/s).  With a the
// scores up to the row's factor, P = a / sum a, q = a / (sum of the chosen):
//   renormalized  x_i = scale q_i (dw_i - sum q dw)     else  x_i = score_i scale dw_i
//   dz_e = P_e (g_e - sum P g) + x_e     (softmax, not renormalized: - P_e sum x)
// and for sigmoid the whole times 1 - sigmoid(z_e).  A row of floats by expert
// in LDS takes the x to the lanes that hold their experts.
template <bool BF, bool BFO, int V, int J, bool SIG>
__global__ __launch_bounds__(64 * kBackWaves) void router_backward_kernel(situ_moe_router_backward_t p, int vec,
                                                                          int vec_out) {
  constexpr int N = V * J;
  __shared__ float rows[kBackWaves][64 * N];
  const int lane = lane_id(), wave = wave_id();
  float* x = rows[wave];
  float g[N];
#pragma unroll
  for (int i = 0; i < N; ++i) { g[i] = 0.0f; x[64 * i + lane] = 0.0f; }
  const bool loss = p.counts != nullptr;
  if (loss) {
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = 64 * V * (i / V) + V * lane + i % V;
      if (e < p.experts) { g[i] = (float)p.counts[e]; c += g[i]; }
    }
    c = wave_sum(c);
    const float f = c > 0.0f ? *p.d_loss * ((float)p.experts * (float)p.top_k) / c / c : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] *= f;
  }
  const int64_t step = (int64_t)gridDim.x * kBackWaves;
  for (int64_t t = (int64_t)blockIdx.x * kBackWaves + wave; t < p.tokens; t += step) {
    const int64_t in = t * p.logits_stride, out = t * p.out_stride;
    float z[N], d[N];
    uint32_t best = 0;
    if (!p.mask || p.mask[t]) {
      load_row<BF, V, J>(p.logits, in, lane, p.experts, vec, z);
#pragma unroll
      for (int i = 0; i < N; ++i) best = max(best, key_of(z[i]));
    }
    const uint32_t top = wave_max(best);
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = 0.0f;
    if (top) {
      const float shift = SIG ? fminf(value_of(top), 0.0f) : value_of(top);
      int id = -1;
      float dw = 0.0f, zc = 0.0f;
      if (p.d_weights && lane < p.top_k) {
        id = p.ids[t * p.top_k + lane];
        if (id >= p.experts) id = -1;
        if (id >= 0) {
          dw = p.d_weights[t * p.top_k + lane] * p.scale;
          zc = load_one<BF>(p.logits, in + id);
        }
      }
      float all = 0.0f, pg = 0.0f;
      scores<SIG, N>(z, shift, d);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        all += d[i];
        pg = fmaf(d[i], g[i], pg);
      }
      const float r = __builtin_amdgcn_rcpf(wave_sum(all));
      pg = loss ? wave_sum(pg) * r : 0.0f;
      if (p.d_weights) {
        float xc;
        if (p.renormalize) {
          const uint32_t topc = wave_max(id >= 0 ? key_of(zc) : 0u);     // of the chosen: they need not be the largest
          const float sc = id >= 0 && topc ? score<SIG>(zc, SIG ? fminf(value_of(topc), 0.0f) : value_of(topc)) : 0.0f;
          const float total = wave_sum(sc);
          const float q = topc ? sc / total : 0.0f;
          xc = q * (dw - wave_sum(q * dw));
        } else {
          xc = id >= 0 ? (SIG ? score<SIG>(zc, 0.0f) : score<SIG>(zc, shift) * r) * dw : 0.0f;
          if constexpr (!SIG) pg += wave_sum(xc);
        }
        if (id >= 0) atomicAdd(&x[id], xc);
        wave_lds();
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = 64 * V * (i / V) + V * lane + i % V;
        d[i] = fmaf(d[i] * r, g[i] - pg, x[e]);
        if constexpr (SIG) {
          const float t1 = e_to(-fabsf(z[i])), o = __builtin_amdgcn_rcpf(1.0f + t1);
          d[i] *= z[i] >= 0.0f ? t1 * o : o;
        }
      }
      wave_lds();
      if (id >= 0) x[id] = 0.0f;
      wave_lds();
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = 64 * V * j + V * lane;
      if constexpr (V == 4) {
        if (vec_out && e + 4 <= p.experts) {
          if constexpr (BFO) {
            const bf16x2 lo = {(__bf16)d[4 * j], (__bf16)d[4 * j + 1]}, hi = {(__bf16)d[4 * j + 2], (__bf16)d[4 * j + 3]};
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.d_logits) + out + e) =
                make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
          } else {
            *reinterpret_cast<f32x4*>(static_cast<float*>(p.d_logits) + out + e) =
                f32x4{d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]};
          }
          continue;
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (e + v < p.experts) {
          if constexpr (BFO)
            static_cast<uint16_t*>(p.d_logits)[out + e + v] = (uint16_t)f32_to_bf16_rne(d[V * j + v]);
          else
            static_cast<float*>(p.d_logits)[out + e + v] = d[V * j + v];
        }
      }
    }
  }
}

template <bool BF, int V, int J, bool SIG, bool BIAS>
void router_go(const RouterArgs& a, int blocks, hipStream_t s) {
  if (a.p.counts)
    hipLaunchKernelGGL((router_kernel<BF, V, J, SIG, BIAS, true>), dim3(blocks), dim3(64 * kRouterWaves), 0, s, a);
  else
    hipLaunchKernelGGL((router_kernel<BF, V, J, SIG, BIAS, false>), dim3(blocks), dim3(64 * kRouterWaves), 0, s, a);
}
template <bool BF, int V, int J>
void router_scored(const RouterArgs& a, int blocks, hipStream_t s) {
  if (a.p.scoring == SITU_SCORE_SOFTMAX) router_go<BF, V, J, false, false>(a, blocks, s);
  else if (!a.p.bias) router_go<BF, V, J, true, false>(a, blocks, s);
  else router_go<BF, V, J, true, true>(a, blocks, s);
}
template <bool BF>
void router_sized(const RouterArgs& a, int blocks, hipStream_t s) {
  const int e = a.p.experts;
  if (e <= 64) router_scored<BF, 1, 1>(a, blocks, s);
  else if (e <= 128) router_scored<BF, 2, 1>(a, blocks, s);
  else if (e <= 256) router_scored<BF, 4, 1>(a, blocks, s);
  else if (e <= 512) router_scored<BF, 4, 2>(a, blocks, s);
  else router_scored<BF, 4, 4>(a, blocks, s);
}

template <bool BF, bool BFO, int V, int J>
void backward_scored(const situ_moe_router_backward_t& p, int vec, int vec_out, int blocks, hipStream_t s) {
  const dim3 grid(blocks), threads(64 * kBackWaves);
  if (p.scoring == SITU_SCORE_SOFTMAX)
    hipLaunchKernelGGL((router_backward_kernel<BF, BFO, V, J, false>), grid, threads, 0, s, p, vec, vec_out);
  else
    hipLaunchKernelGGL((router_backward_kernel<BF, BFO, V, J, true>), grid, threads, 0, s, p, vec, vec_out);
}
template <bool BF, bool BFO>
void backward_sized(const situ_moe_router_backward_t& p, int vec, int vec_out, int blocks, hipStream_t s) {
  const int e = p.experts;
  if (e <= 64) backward_scored<BF, BFO, 1, 1>(p, vec, vec_out, blocks, s);
  else if (e <= 128) backward_scored<BF, BFO, 2, 1>(p, vec, vec_out, blocks, s);
  else if (e <= 256) backward_scored<BF, BFO, 4, 1>(p, vec, vec_out, blocks, s);
  else if (e <= 512) backward_scored<BF, BFO, 4, 2>(p, vec, vec_out, blocks, s);
  else backward_scored<BF, BFO, 4, 4>(p, vec, vec_out, blocks, s);
}

// Whether every row's experts can be moved four (two up to 128 experts) at a time.
int at_once(const void* p, int64_t stride, bool bf, int experts) {
  const int v = experts <= 128 ? 2 : 4;
  return reinterpret_cast<uintptr_t>(p) % (unsigned)(bf ? 2 * v : 4 * v) == 0 && stride % v == 0;
}

}  // namespace

int router_blocks(int32_t tokens) {
  return tokens <= kOneBlockTokens ? 1 : std::min(kRouterBlocks, (tokens + kRouterWaves - 1) / kRouterWaves);
}

hipError_t launch_router(const situ_moe_router_t& p, hipStream_t s) {
  RouterArgs a{};
  a.p = p;
  const bool bf = p.logits_dtype == SITU_OUT_BF16;
  a.vec = at_once(p.logits, p.logits_stride, bf, p.experts);
  const bool balance = p.counts != nullptr;
  // Without the loss, more workgroups (32768 x 256, sigmoid and bias: 1536 23.1 us, 768 23.7, 1024 24.5, 4096 26.6).
  // With it and a bias, the rows of over 512 experts leave LDS for two workgroups a CU (32768 x 896: 512 52.6 us, 768 58).
  const int groups = (p.tokens + kRouterWaves - 1) / kRouterWaves;
  const int blocks = !balance                       ? std::min(groups, 2 * kRouterBlocks)
                     : p.bias && p.experts > 512 ? std::min(router_blocks(p.tokens), 512)
                                                 : router_blocks(p.tokens);
  if (balance && blocks > 1) {
    const int64_t part = (int64_t)blocks * p.experts;
    a.part_sum = static_cast<float*>(p.workspace);
    a.part_count = reinterpret_cast<int32_t*>(a.part_sum + part);
    a.ticket = reinterpret_cast<uint32_t*>(a.part_count + part);
  }
  if (bf) router_sized<true>(a, blocks, s);
  else router_sized<false>(a, blocks, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !balance || blocks == 1) return e;
  const dim3 grid((p.experts + kFinishExperts - 1) / kFinishExperts);
  hipLaunchKernelGGL(router_finish_kernel, grid, dim3(64 * kFinishWaves), 0, s, a, blocks);
  return hipGetLastError();
}

hipError_t launch_router_backward(const situ_moe_router_backward_t& p, hipStream_t s) {
  const bool bf = p.logits_dtype == SITU_OUT_BF16, bfo = p.out_dtype == SITU_OUT_BF16;
  const int vec = at_once(p.logits, p.logits_stride, bf, p.experts);
  const int vec_out = at_once(p.d_logits, p.out_stride, bfo, p.experts);
  const int blocks = (int)std::min<int64_t>(((int64_t)p.tokens + kBackWaves - 1) / kBackWaves, kBackBlocks);
  if (bf) {
    if (bfo) backward_sized<true, true>(p, vec, vec_out, blocks, s);
    else backward_sized<true, false>(p, vec, vec_out, blocks, s);
  } else {
    if (bfo) backward_sized<false, true>(p, vec, vec_out, blocks, s);
    else backward_sized<false, false>(p, vec, vec_out, blocks, s);
  }
  return hipGetLastError();
}

}  // namespace situ
