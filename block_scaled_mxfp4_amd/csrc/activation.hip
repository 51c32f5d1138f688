// The gated activation between the expert products, with gate and up kept in 8
// bits for the way back, and its gradient (situ_moe_activation,
// situ_moe_activation_backward).
//
// With t = tanh, s the sigmoid:
//   SiTU        h = b t(g/b) s(g) l t(u/l)
//               dg = dh (t'(g/b) s(g) + b t(g/b) s(g) s(-g)) l t(u/l)    du = dh b t(g/b) s(g) t'(u/l)
//   SwiGLU, SwigluBias (a = 1, c = 0 without)
//               h = g s(a g) (u + c)
//               dg = dh s(a g) (1 + a g s(-a g)) (u + c)                 du = dh g s(a g)
// t' = 1 - t^2 = 4 e / (1 + e)^2 with e = e^-2|x|, and s(-x) from the same
// exponential as s(x): neither is a difference of near numbers.
//
// Elementwise: 8 bytes a (gate, up) pair forward with codes, 10 backward from codes
// with h.  Forward with codes the vector units' issue binds as much as HBM does:
// 262144 x 384 is 56 slots a pair, 145 us of the SIMDs at 2.4 GHz and 165 at 2.1,
// beside 165 us of the bytes at the 4.9 TB/s of a large copy.  It takes 152 to 166 us,
// by the clock that the card holds, and has taken 189 for some ten milliseconds
// after a pause.  The gradient, 65521 x 768, is bound by HBM: 102 to 109 us (4.8
// TB/s), 124 in such a stretch.  Sixteen lanes take 128 columns of a row's gate and
// the same of its up, eight each (16 bytes): a block of the 8-bit format, whose
// maximum is then four DPP moves.  They walk the row's blocks, so that the row's
// expert is looked up once, in LDS, where the offsets and constants are copied.
#include <algorithm>

#include "quant_block.hpp"
#include "routed.hpp"

namespace situ {

namespace {

constexpr float kL2e = 1.44269502162933349609375f;   // log2(e) rounded to fp32
constexpr int kActThreads = 256;
constexpr int kRows = kActThreads / 16;               // rows a workgroup takes at once
constexpr int kActExperts = 1024;

struct ActArgs {
  situ_moe_activation_t p;
  int32_t blocks;             // of 128 columns a row
  int32_t run;                // of them that sixteen lanes walk
  int32_t share;              // rows of a workgroup, consecutive
};

// Constants of a row.
struct RowK {
  float b, ib, l, il;         // SiTU: |beta|, 1 / |beta|, |linear beta| and its inverse; else b = a, l = c
};
// b t(x/b) is even in b and, from |b| = 2^123 on, x for every |x| up to 2^111: larger ones (infinity too) are taken for
// 2^123, so that nothing leaves fp32's range before h does (below) and 1 / b is a normal value.  NaN stays.
__device__ __forceinline__ void saturation(float b, float& limit, float& inverse) {
  limit = __builtin_elementwise_minimum(fabsf(b), 0x1p123f);
  inverse = __builtin_elementwise_minimum(__builtin_amdgcn_rcpf(limit), 0x1p126f);
}

struct Experts {
  int32_t offsets[kActExperts + 1];
  float p0[kActExperts], p1[kActExperts];
};
__device__ __forceinline__ void load_experts(Experts& x, const situ_moe_activation_t& p, bool constants) {
  for (int i = threadIdx.x; i < p.experts; i += kActThreads) {
    x.offsets[i] = p.offsets ? p.offsets[i] : 0;
    if (constants) { x.p0[i] = p.p0[i]; x.p1[i] = p.p1[i]; }
  }
  if (threadIdx.x == 0) x.offsets[p.experts] = p.offsets ? p.offsets[p.experts] : p.rows;
  __syncthreads();
}
// The expert e of a row: the last one that starts at or before it (its group then holds the row, where any does).  The
// rows of a thread ascend, so that all but the first search (e < 0) go on from the row before.
__device__ __forceinline__ bool find_expert(const Experts& x, int experts, int row, int& e) {
  if (row < x.offsets[0] || row >= x.offsets[experts]) return false;
  if (e < 0) {
    int hi = experts;
    e = 0;
    while (hi - e > 1) {
      const int mid = (e + hi) / 2;
      if (x.offsets[mid] <= row) e = mid; else hi = mid;
    }
  }
  while (e + 1 < experts && x.offsets[e + 1] <= row) ++e;
  return true;
}
template <int KIND>
__device__ __forceinline__ RowK row_k(const Experts& x, int e) {
  if constexpr (KIND == SITU_ACTIVATION_SWIGLU) return RowK{1.0f, 1.0f, 0.0f, 1.0f};
  if constexpr (KIND == SITU_ACTIVATION_SWIGLU_BIAS) return RowK{x.p0[e], 1.0f, x.p1[e], 1.0f};
  RowK k;
  saturation(x.p0[e], k.b, k.ib);
  saturation(x.p1[e], k.l, k.il);
  return k;
}

// b tanh(x / b) = n / d of fp32 values: x clamped to 8 b (tanh(8) is 1 - 2^-22), c = x / b, n = x P(c^2), d = Q(c^2) with
// P of degree 3 and Q of 4, fitted on [0, 8] for the smallest largest relative error (reweighted least squares on the
// linearized residual c P - tanh(c) Q): 1.5e-7, within 6 * 2^-24 as evaluated here.  With x and not c in n, no b is
// multiplied back: the value is right where c underflows.  Both are divided by 2^E.  Q lies in [1, 195.2]: with E of 12
// for gate and 4 for up the product of their d, at most 0.59, and 1 + e^-g overflows no sooner than e^-g does, and its
// reciprocal is a normal value where e^-g is up to 2^126; for |b| and |l| up to 2^123 gate times the reciprocal, h / (l t3
// d3), is below 2^128, and so is l t3 d3.  A NaN stays one.
template <int E>
__device__ __forceinline__ void tanh_parts(float x, float b, float inverse, float& n, float& d) {
  constexpr float k = 1.0f / (1 << E);
  x = __builtin_elementwise_maximum(__builtin_elementwise_minimum(x, 8.0f * b), -8.0f * b);
  const float c = x * inverse, s = c * c;
  float p = 1.1475112e-05f * k, q = 2.4732324e-07f * k;
  q = fmaf(q, s, 0.000239314897f * k);
  p = fmaf(p, s, 0.00295580747f * k);  q = fmaf(q, s, 0.0238357844f * k);
  p = fmaf(p, s, 0.129303546f * k);    q = fmaf(q, s, 0.462636088f * k);
  p = fmaf(p, s, k);                   q = fmaf(q, s, k);
  n = x * p;
  d = q;
}

template <int KIND>
__device__ __forceinline__ float act(float g, float u, const RowK& k) {
  if constexpr (KIND == SITU_ACTIVATION_SITU) {
    float n1, d1, n3, d3;
    tanh_parts<12>(g, k.b, k.ib, n1, d1);
    tanh_parts<4>(u, k.l, k.il, n3, d3);
    const float e = __builtin_amdgcn_exp2f(g * -kL2e), t = d1 * d3;
    return n1 * __builtin_amdgcn_rcpf(fmaf(t, e, t)) * n3;      // the factor that may be 0 first: n1 n3 may overflow
  } else {
    const float e = __builtin_amdgcn_exp2f(k.b * g * -kL2e);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * (u + k.l);      // the small factor first: g u may overflow
  }
}

// b t and 1 - t^2 = (1 - t)(1 + t) for t = tanh(x), x = v / b, with e = e^-2|x|: t = 1 - e r and 1 + t = r, r = 2 / (1 + e).
// Below 1/16, where 1 - e r is a difference of near numbers, the odd series to x^5 (v times its even part: v may be where
// x underflows), off by less than 2^-27; above it 1 - e r is within 2^-20 of its value.
__device__ __forceinline__ void tanh_slope(float v, float b, float inverse, float& bt, float& slope) {
  const float x = v * inverse;
  const float e = __builtin_amdgcn_exp2f(fabsf(x) * (-2.0f * kL2e));
  const float r = __builtin_amdgcn_rcpf(fmaf(e, 0.5f, 0.5f)), er = e * r;
  slope = er * r;
  const float x2 = x * x;
  const float series = v * fmaf(x2, fmaf(x2, 2.0f / 15.0f, -1.0f / 3.0f), 1.0f);
  bt = fabsf(x) < 0.0625f ? series : __builtin_copysignf(fmaf(-b, er, b), v);
}
__device__ __forceinline__ void sigmoid_both(float x, float& s, float& left) {
  const float e = __builtin_amdgcn_exp2f(fabsf(x) * -kL2e);
  const float r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
  s = x < 0.0f ? er : r;
  left = x < 0.0f ? r : er;
}

template <int KIND>
__device__ __forceinline__ void act_backward(float g, float u, float dh, const RowK& k, float& dg, float& du, float& h) {
  if constexpr (KIND == SITU_ACTIVATION_SITU) {
    float gate, s1, up, s3, s, left;
    tanh_slope(g, k.b, k.ib, gate, s1);
    tanh_slope(u, k.l, k.il, up, s3);
    sigmoid_both(g, s, left);
    gate *= s;
    h = gate * up;
    dg = dh * (up * fmaf(gate, left, s1 * s));       // the factor is at most 1.1, and dh up may overflow where it is 0
    du = dh * (gate * s3);
  } else {
    float s, left;
    float x = k.b * g;
    // an overflow to infinity would meet a factor of 0; s is 0 or 1 from 2^7 on.  A NaN stays one
    if constexpr (KIND == SITU_ACTIVATION_SWIGLU_BIAS)
      x = __builtin_elementwise_maximum(__builtin_elementwise_minimum(x, 0x1p20f), -0x1p20f);
    sigmoid_both(x, s, left);
    const float gate = g * s, up = u + k.l;
    h = gate * up;
    dg = dh * (s * fmaf(x, left, 1.0f)) * up;
    du = dh * gate;
  }
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
__device__ __forceinline__ void codes8(const uint2& c, float s, float f[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int w = (int)(i ? c.y : c.x);
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    f[4 * i] = lo[0] * s;
    f[4 * i + 1] = lo[1] * s;
    f[4 * i + 2] = hi[0] * s;
    f[4 * i + 3] = hi[1] * s;
  }
}
// The largest magnitude of the sixteen lanes' eight (a NaN is passed over).
template <int kCtrl>
__device__ __forceinline__ float row_max(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xf, 0xf, true);
  return fmaxf(v, __builtin_bit_cast(float, o));
}
__device__ __forceinline__ float amax16(const float f[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) m = fmaxf(fmaxf(fabsf(f[i]), fabsf(f[i + 1])), m);
  m = row_max<0x128>(m);
  m = row_max<0x124>(m);
  m = row_max<0x122>(m);
  return row_max<0x121>(m);
}

// Codes pass the caches by: they are read on the way back (262144 x 384: 213 us stored as h is, 189 so).
__device__ __forceinline__ void put(uint8_t* p, const uint2& v) {
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  __builtin_nontemporal_store(i32x2{(int)v.x, (int)v.y}, reinterpret_cast<i32x2*>(p));
}

// gate_up is read once (262144 x 384, the least of each: 168 us with ordinary loads, 150 so; the gradient's inputs gained
// nothing by it).
__device__ __forceinline__ uint4 load_once(const uint16_t* p) {
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(p)));
}

template <int KIND, bool KEEP>
__global__ __launch_bounds__(kActThreads) void activation_kernel(ActArgs a) {
  __shared__ Experts x;
  const situ_moe_activation_t& p = a.p;
  load_experts(x, p, KIND != SITU_ACTIVATION_SWIGLU);
  const int at = threadIdx.x & 15;
  // this workgroup's rows, sixteen at a time, and columns
  const int first = blockIdx.y * a.run, last = min(first + a.run, a.blocks);
  const int end = (int)min((int64_t)(blockIdx.x + 1) * a.share, (int64_t)p.rows);
  int row = (int)(blockIdx.x * a.share) + (int)(threadIdx.x / 16), e = -1;
  const uint16_t* gu = p.gate_up + (int64_t)row * p.gate_up_stride + 8 * at;
  uint16_t* h = p.h + (int64_t)row * p.h_stride + 8 * at;
  uint8_t* codes = p.codes + (int64_t)row * (2 * p.inner) + 8 * at;
  float* scales = p.scales + (int64_t)row * (2 * a.blocks);
  for (; row < end; row += kRows, gu += kRows * p.gate_up_stride, h += kRows * p.h_stride,
                    codes += (int64_t)kRows * 2 * p.inner, scales += kRows * 2 * a.blocks) {
    if (!find_expert(x, p.experts, row, e)) continue;
    const RowK k = row_k<KIND>(x, e);
    for (int b = first; b < last; ++b) {
      const int col = b * 128;
      const bool in = col + 8 * at < p.inner;
      float g[8], u[8], o[8];
      uint4 vg = make_uint4(0, 0, 0, 0), vu = vg;
      if (in) {
        vg = load_once(gu + col);
        vu = load_once(gu + p.inner + col);
      }
      unpack8(vg, g);
      unpack8(vu, u);
      if constexpr (KEEP) {
        const float sg = block_scale(amax16(g)), su = block_scale(amax16(u));
        if (in) {
          put(codes + col, block_codes(g, sg));
          put(codes + p.inner + col, block_codes(u, su));
        }
        if (at == 0) {
          scales[b] = sg;
          scales[a.blocks + b] = su;
        }
      }
      if (in) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = act<KIND>(g[i], u[i], k);
        *reinterpret_cast<uint4*>(h + col) = pack8(o);
      }
    }
  }
}

template <int KIND, bool KEPT, bool AGAIN>
__global__ __launch_bounds__(kActThreads) void activation_backward_kernel(ActArgs a) {
  __shared__ Experts x;
  const situ_moe_activation_t& p = a.p;
  load_experts(x, p, KIND != SITU_ACTIVATION_SWIGLU);
  const int at = threadIdx.x & 15;
  const int first = blockIdx.y * a.run, last = min(first + a.run, a.blocks);
  const int end = (int)min((int64_t)(blockIdx.x + 1) * a.share, (int64_t)p.rows);
  int row = (int)(blockIdx.x * a.share) + (int)(threadIdx.x / 16), e = -1;
  const uint16_t* gu = p.gate_up + (int64_t)row * p.gate_up_stride + 8 * at;
  const uint16_t* dhs = p.dh + (int64_t)row * p.dh_stride + 8 * at;
  const uint8_t* codes = p.codes + (int64_t)row * (2 * p.inner) + 8 * at;
  const float* scales = p.scales + (int64_t)row * (2 * a.blocks);
  uint16_t* hs = p.h + (int64_t)row * p.h_stride + 8 * at;
  uint16_t* ds = p.d_gate_up + (int64_t)row * p.d_gate_up_stride + 8 * at;
  for (; row < end; row += kRows, gu += kRows * p.gate_up_stride, dhs += kRows * p.dh_stride,
                    codes += (int64_t)kRows * 2 * p.inner, scales += kRows * 2 * a.blocks, hs += kRows * p.h_stride,
                    ds += kRows * p.d_gate_up_stride) {
    if (!find_expert(x, p.experts, row, e)) continue;
    const RowK k = row_k<KIND>(x, e);
    for (int b = first; b < last; ++b) {
      const int col = b * 128;
      if (col + 8 * at >= p.inner) continue;
      float g[8], u[8], dh[8], h[8];
      if constexpr (KEPT) {
        const uint2 cg = *reinterpret_cast<const uint2*>(codes + col);
        const uint2 cu = *reinterpret_cast<const uint2*>(codes + p.inner + col);
        codes8(cg, scales[b], g);
        codes8(cu, scales[a.blocks + b], u);
      } else {
        unpack8(*reinterpret_cast<const uint4*>(gu + col), g);
        unpack8(*reinterpret_cast<const uint4*>(gu + p.inner + col), u);
      }
      unpack8(*reinterpret_cast<const uint4*>(dhs + col), dh);
#pragma unroll
      for (int i = 0; i < 8; ++i) act_backward<KIND>(g[i], u[i], dh[i], k, g[i], u[i], h[i]);
      *reinterpret_cast<uint4*>(ds + col) = pack8(g);
      *reinterpret_cast<uint4*>(ds + p.inner + col) = pack8(u);
      if constexpr (AGAIN) *reinterpret_cast<uint4*>(hs + col) = pack8(h);
    }
  }
}

// Sixteen lanes walk a whole row where there are rows enough for 32 waves a CU, and parts of one where there are not.
// With many rows a CU gets 32 workgroups' shares in turn, so that what is moved at one time lies together (262144 x 384:
// 176 us with one share each, 168 with four), but not more, as each copies the experts' constants.
ActArgs act_args(const situ_moe_activation_t& p, int cus, dim3& grid) {
  ActArgs a{};
  a.p = p;
  a.blocks = (p.inner + 127) / 128;
  const int wanted = cus * 8;                        // workgroups at once
  const int groups = (p.rows + kRows - 1) / kRows;
  const int runs = std::min(a.blocks, std::max(1, wanted / groups));
  a.run = (a.blocks + runs - 1) / runs;
  grid.y = (unsigned)((a.blocks + a.run - 1) / a.run);
  const int shares = std::min(groups, std::max(1, 4 * wanted / (int)grid.y));
  a.share = (groups + shares - 1) / shares * kRows;
  grid.x = (unsigned)((p.rows + a.share - 1) / a.share);
  return a;
}

template <int KIND>
void forward_go(const ActArgs& a, dim3 grid, hipStream_t s) {
  if (a.p.codes) hipLaunchKernelGGL((activation_kernel<KIND, true>), grid, dim3(kActThreads), 0, s, a);
  else hipLaunchKernelGGL((activation_kernel<KIND, false>), grid, dim3(kActThreads), 0, s, a);
}
template <int KIND, bool KEPT>
void backward_go(const ActArgs& a, dim3 grid, hipStream_t s) {
  if (a.p.h) hipLaunchKernelGGL((activation_backward_kernel<KIND, KEPT, true>), grid, dim3(kActThreads), 0, s, a);
  else hipLaunchKernelGGL((activation_backward_kernel<KIND, KEPT, false>), grid, dim3(kActThreads), 0, s, a);
}

}  // namespace

hipError_t launch_activation(const situ_moe_activation_t& p, int cus, hipStream_t s) {
  dim3 grid;
  const ActArgs a = act_args(p, cus, grid);
  switch (p.activation) {
    case SITU_ACTIVATION_SITU: forward_go<SITU_ACTIVATION_SITU>(a, grid, s); break;
    case SITU_ACTIVATION_SWIGLU: forward_go<SITU_ACTIVATION_SWIGLU>(a, grid, s); break;
    default: forward_go<SITU_ACTIVATION_SWIGLU_BIAS>(a, grid, s); break;
  }
  return hipGetLastError();
}

hipError_t launch_activation_backward(const situ_moe_activation_t& p, int cus, hipStream_t s) {
  dim3 grid;
  const ActArgs a = act_args(p, cus, grid);
  const bool kept = !p.gate_up;
  switch (p.activation) {
    case SITU_ACTIVATION_SITU:
      if (kept) backward_go<SITU_ACTIVATION_SITU, true>(a, grid, s);
      else backward_go<SITU_ACTIVATION_SITU, false>(a, grid, s);
      break;
    case SITU_ACTIVATION_SWIGLU:
      if (kept) backward_go<SITU_ACTIVATION_SWIGLU, true>(a, grid, s);
      else backward_go<SITU_ACTIVATION_SWIGLU, false>(a, grid, s);
      break;
    default:
      if (kept) backward_go<SITU_ACTIVATION_SWIGLU_BIAS, true>(a, grid, s);
      else backward_go<SITU_ACTIVATION_SWIGLU_BIAS, false>(a, grid, s);
      break;
  }
  return hipGetLastError();
}

}  // namespace situ
