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
// Elementwise, bound by HBM: 8 bytes a (gate, up) pair forward with codes, as
// many backward from codes.  Sixteen lanes take 128 columns of a row's gate and
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
constexpr int kActExperts = 1024;

struct ActArgs {
  situ_moe_activation_t p;
  int32_t blocks;             // of 128 columns a row
  int32_t run;                // of them that sixteen lanes walk
  int32_t runs;               // of them a row
  int64_t items;              // rows * runs
};

// Constants of a row.
struct RowK {
  float b, ib, l, il;         // SiTU: beta, 1 / beta, linear beta and its inverse; else b = a, l = c
};

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
// The expert of a row, -1 outside every group: the last one that starts at or before it, where it also ends behind it.
__device__ __forceinline__ int expert_of(const Experts& x, int experts, int row) {
  int lo = 0, hi = experts;   // offsets[lo] <= row < offsets[hi], if any
  if (row < x.offsets[0] || row >= x.offsets[experts]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (x.offsets[mid] <= row) lo = mid; else hi = mid;
  }
  return lo;
}
template <int KIND>
__device__ __forceinline__ RowK row_k(const Experts& x, int e) {
  if constexpr (KIND == SITU_ACTIVATION_SWIGLU) return RowK{1.0f, 1.0f, 0.0f, 1.0f};
  const float b = x.p0[e], l = x.p1[e];
  return RowK{b, 1.0f / b, l, 1.0f / l};
}

// tanh_nd (common.hpp) for any x: a NaN stays one.
__device__ __forceinline__ void tanh_parts(float x, float& n, float& d) {
  tanh_nd(x, n, d);
  n = x != x ? x : n;
}

template <int KIND>
__device__ __forceinline__ float act(float g, float u, const RowK& k) {
  if constexpr (KIND == SITU_ACTIVATION_SITU) {
    float n1, d1, n3, d3;
    tanh_parts(g * k.ib, n1, d1);
    tanh_parts(u * k.il, n3, d3);
    // sigmoid = 1 / (1 + e), or e / (1 + e) for g < 0: no exponential that overflows
    const float e = __builtin_amdgcn_exp2f(-fabsf(g) * kL2e), t = d1 * d3;
    return (n1 * n3) * (g < 0.0f ? e : 1.0f) * __builtin_amdgcn_rcpf(fmaf(t, e, t)) * (k.b * k.l);
  } else {
    const float x = k.b * g, e = __builtin_amdgcn_exp2f(-fabsf(x) * kL2e);
    return g * (u + k.l) * (x < 0.0f ? e : 1.0f) * __builtin_amdgcn_rcpf(1.0f + e);
  }
}

// tanh(x) and 1 - tanh(x)^2.  Below 1/4 the quotient would be a difference of near numbers: the odd series
// to x^9, off by less than 2^-24 there.
__device__ __forceinline__ void tanh_slope(float x, float& t, float& slope) {
  const float e = __builtin_amdgcn_exp2f(fabsf(x) * (-2.0f * kL2e));
  const float r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
  slope = 4.0f * er * r;
  const float x2 = x * x;
  float q = fmaf(x2, 62.0f / 2835.0f, -17.0f / 315.0f);
  q = fmaf(x2, q, 2.0f / 15.0f);
  q = fmaf(x2, q, -1.0f / 3.0f);
  const float series = fmaf(x2 * x, q, x);
  t = fabsf(x) < 0.25f ? series : __builtin_copysignf(fmaf(-2.0f, er, 1.0f), x);
}
__device__ __forceinline__ void sigmoid_both(float x, float& s, float& left) {
  const float e = __builtin_amdgcn_exp2f(-fabsf(x) * kL2e);
  const float r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
  s = x < 0.0f ? er : r;
  left = x < 0.0f ? r : er;
}

template <int KIND>
__device__ __forceinline__ void act_backward(float g, float u, float dh, const RowK& k, float& dg, float& du, float& h) {
  if constexpr (KIND == SITU_ACTIVATION_SITU) {
    float t1, s1, t3, s3, s, left;
    tanh_slope(g * k.ib, t1, s1);
    tanh_slope(u * k.il, t3, s3);
    sigmoid_both(g, s, left);
    const float gate = k.b * t1 * s, up = k.l * t3;
    h = gate * up;
    dg = dh * up * fmaf(gate, left, s1 * s);
    du = dh * gate * s3;
  } else {
    float s, left;
    const float x = k.b * g;
    sigmoid_both(x, s, left);
    const float gate = g * s, up = u + k.l;
    h = gate * up;
    dg = dh * up * (s * fmaf(x, left, 1.0f));
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
    f[4 * i] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * s;
    f[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * s;
    f[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * s;
    f[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * s;
  }
}
// The largest magnitude of the sixteen lanes' eight (a NaN is passed over).
template <int kCtrl>
__device__ __forceinline__ float row_max(float v) {
  return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xf, 0xf, true)));
}
__device__ __forceinline__ float amax16(const float f[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  m = row_max<0x128>(m);
  m = row_max<0x124>(m);
  m = row_max<0x122>(m);
  return row_max<0x121>(m);
}

template <int KIND, bool KEEP>
__global__ __launch_bounds__(kActThreads) void activation_kernel(ActArgs a) {
  __shared__ Experts x;
  const situ_moe_activation_t& p = a.p;
  load_experts(x, p, KIND != SITU_ACTIVATION_SWIGLU);
  const int at = threadIdx.x & 15;
  for (int64_t item = (int64_t)blockIdx.x * (kActThreads / 16) + threadIdx.x / 16; item < a.items;
       item += (int64_t)gridDim.x * (kActThreads / 16)) {
    const int row = (int)((uint32_t)item / (uint32_t)a.runs), first = (int)((uint32_t)item - (uint32_t)row * a.runs) * a.run;
    const int e = expert_of(x, p.experts, row);
    if (e < 0) continue;
    const RowK k = row_k<KIND>(x, e);
    const uint16_t* gu = p.gate_up + (int64_t)row * p.gate_up_stride;
    for (int b = first; b < min(first + a.run, a.blocks); ++b) {
      const int col = b * 128 + 8 * at;
      const bool in = col < p.inner;
      float g[8], u[8];
      uint4 vg = make_uint4(0, 0, 0, 0), vu = vg;
      if (in) {
        vg = *reinterpret_cast<const uint4*>(gu + col);
        vu = *reinterpret_cast<const uint4*>(gu + p.inner + col);
      }
      unpack8(vg, g);
      unpack8(vu, u);
      if constexpr (KEEP) {
        const float sg = block_scale(amax16(g)), su = block_scale(amax16(u));
        if (in) {
          uint8_t* c = p.codes + (int64_t)row * (2 * p.inner) + col;
          *reinterpret_cast<uint2*>(c) = block_codes(g, sg);
          *reinterpret_cast<uint2*>(c + p.inner) = block_codes(u, su);
        }
        if (at == 0) {
          float* s = p.scales + (int64_t)row * (2 * a.blocks) + b;
          s[0] = sg;
          s[a.blocks] = su;
        }
      }
      if (in) {
        float h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = act<KIND>(g[i], u[i], k);
        *reinterpret_cast<uint4*>(p.h + (int64_t)row * p.h_stride + col) = pack8(h);
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
  for (int64_t item = (int64_t)blockIdx.x * (kActThreads / 16) + threadIdx.x / 16; item < a.items;
       item += (int64_t)gridDim.x * (kActThreads / 16)) {
    const int row = (int)((uint32_t)item / (uint32_t)a.runs), first = (int)((uint32_t)item - (uint32_t)row * a.runs) * a.run;
    const int e = expert_of(x, p.experts, row);
    if (e < 0) continue;
    const RowK k = row_k<KIND>(x, e);
    for (int b = first; b < min(first + a.run, a.blocks); ++b) {
      const int col = b * 128 + 8 * at;
      if (col >= p.inner) continue;
      float g[8], u[8], dh[8], h[8];
      if constexpr (KEPT) {
        const uint8_t* c = p.codes + (int64_t)row * (2 * p.inner) + col;
        const float* s = p.scales + (int64_t)row * (2 * a.blocks) + b;
        const uint2 cg = *reinterpret_cast<const uint2*>(c), cu = *reinterpret_cast<const uint2*>(c + p.inner);
        codes8(cg, s[0], g);
        codes8(cu, s[a.blocks], u);
      } else {
        const uint16_t* gu = p.gate_up + (int64_t)row * p.gate_up_stride + col;
        unpack8(*reinterpret_cast<const uint4*>(gu), g);
        unpack8(*reinterpret_cast<const uint4*>(gu + p.inner), u);
      }
      unpack8(*reinterpret_cast<const uint4*>(p.dh + (int64_t)row * p.dh_stride + col), dh);
#pragma unroll
      for (int i = 0; i < 8; ++i) act_backward<KIND>(g[i], u[i], dh[i], k, g[i], u[i], h[i]);
      uint16_t* d = p.d_gate_up + (int64_t)row * p.d_gate_up_stride + col;
      *reinterpret_cast<uint4*>(d) = pack8(g);
      *reinterpret_cast<uint4*>(d + p.inner) = pack8(u);
      if constexpr (AGAIN) *reinterpret_cast<uint4*>(p.h + (int64_t)row * p.h_stride + col) = pack8(h);
    }
  }
}

// Sixteen lanes walk a whole row where there are rows enough for 32 waves a CU,
// and parts of one where there are not.
ActArgs act_args(const situ_moe_activation_t& p, int cus) {
  ActArgs a{};
  a.p = p;
  a.blocks = (p.inner + 127) / 128;
  const int64_t wanted = (int64_t)cus * 32 * 4;
  const int64_t runs = std::min<int64_t>(a.blocks, std::max<int64_t>(1, wanted / std::max(p.rows, 1)));
  a.run = (int)((a.blocks + runs - 1) / runs);
  a.runs = (a.blocks + a.run - 1) / a.run;
  a.items = (int64_t)p.rows * a.runs;
  return a;
}
int act_grid(const ActArgs& a, int cus) {
  constexpr int kItems = kActThreads / 16;
  return (int)std::min<int64_t>((a.items + kItems - 1) / kItems, (int64_t)cus * 8);
}

template <int KIND>
void forward_go(const ActArgs& a, int grid, hipStream_t s) {
  if (a.p.codes) hipLaunchKernelGGL((activation_kernel<KIND, true>), dim3(grid), dim3(kActThreads), 0, s, a);
  else hipLaunchKernelGGL((activation_kernel<KIND, false>), dim3(grid), dim3(kActThreads), 0, s, a);
}
template <int KIND, bool KEPT>
void backward_go(const ActArgs& a, int grid, hipStream_t s) {
  if (a.p.h) hipLaunchKernelGGL((activation_backward_kernel<KIND, KEPT, true>), dim3(grid), dim3(kActThreads), 0, s, a);
  else hipLaunchKernelGGL((activation_backward_kernel<KIND, KEPT, false>), dim3(grid), dim3(kActThreads), 0, s, a);
}

}  // namespace

hipError_t launch_activation(const situ_moe_activation_t& p, int cus, hipStream_t s) {
  const ActArgs a = act_args(p, cus);
  const int grid = act_grid(a, cus);
  switch (p.activation) {
    case SITU_ACTIVATION_SITU: forward_go<SITU_ACTIVATION_SITU>(a, grid, s); break;
    case SITU_ACTIVATION_SWIGLU: forward_go<SITU_ACTIVATION_SWIGLU>(a, grid, s); break;
    default: forward_go<SITU_ACTIVATION_SWIGLU_BIAS>(a, grid, s); break;
  }
  return hipGetLastError();
}

hipError_t launch_activation_backward(const situ_moe_activation_t& p, int cus, hipStream_t s) {
  const ActArgs a = act_args(p, cus);
  const int grid = act_grid(a, cus);
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
