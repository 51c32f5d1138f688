// Entry points of the products grouped by expert and of the E4M3 products
// with scales per 128: argument checks, then one launch each (or the name of
// the kernel that would be launched).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/situ_moe.h"
#include "checks.hpp"
#include "grouped.hpp"
#include "internal.hpp"

namespace {

using situ::aligned;
using situ::check_in;
using situ::check_out;
using situ::fail_status;
using situ::launched;

constexpr int32_t kMaxRows = 1 << 24, kMaxSide = 1 << 18, kMaxExperts = 1024;
constexpr int64_t kMaxScaleStride = 1 << 22;   // 64 rows of scales within 32 bits of bytes

situ_status check_sizes(int32_t rows, int32_t n, int32_t k, int32_t experts, int32_t out_dtype, int32_t reserved,
                        const int32_t* offsets) {
  if (rows < 0 || n < 1 || k < 1 || experts < 1)
    return fail_status(SITU_E_BAD_SHAPE, "rows %d, n %d, k %d, experts %d", rows, n, k, experts);
  if (rows > kMaxRows || n > kMaxSide || k > kMaxSide || experts > kMaxExperts)
    return fail_status(SITU_E_UNSUPPORTED, "rows %d (at most 2^24), n %d, k %d (2^18), experts %d (1024)", rows, n, k,
                       experts);
  if (out_dtype != SITU_OUT_F32 && out_dtype != SITU_OUT_BF16)
    return fail_status(SITU_E_UNSUPPORTED, "out_dtype %d", out_dtype);
  if (reserved != 0) return fail_status(SITU_E_BAD_SHAPE, "reserved is %d, not 0", reserved);
  if (!offsets && experts != 1) return fail_status(SITU_E_NULL_ARG, "offsets is NULL with %d experts", experts);
  if (!aligned(offsets, 4)) return fail_status(SITU_E_BAD_SHAPE, "offsets must be 4-byte aligned");
  return SITU_OK;
}

// Checks the arguments and fills in the kernels'; `nothing`: there is nothing to compute.
situ_status grouped_args(situ::GroupedMode mode, const situ_moe_grouped_t* p, situ::GroupedArgs& a, bool& nothing) {
  nothing = false;
  if (!p) return fail_status(SITU_E_NULL_ARG, "args is NULL");
  situ_status st = check_sizes(p->rows, p->n, p->k, p->experts, p->out_dtype, p->reserved, p->offsets);
  if (st != SITU_OK) return st;
  const bool fwd = mode == situ::kGFwd, wgrad = mode == situ::kGWgrad;
  if (p->k % 8 || (!fwd && p->n % 8))
    return fail_status(SITU_E_BAD_SHAPE, "k %d%s must be a multiple of 8", p->k, fwd ? "" : " and n");
  if (p->x_div < 0 || p->y_div < 0 || (fwd && p->y_div > 1) || (mode == situ::kGDgrad && p->x_div > 1))
    return fail_status(SITU_E_BAD_SHAPE, "x_div %d, y_div %d (0 or 1 on the written side)", p->x_div, p->y_div);
  const bool indexed = p->x_div || p->y_div;
  if (indexed && !p->pairs && p->rows > 0) return fail_status(SITU_E_NULL_ARG, "pairs is NULL");
  if (!aligned(p->pairs, 4)) return fail_status(SITU_E_BAD_SHAPE, "pairs must be 4-byte aligned");
  if ((p->x_div && p->x_rows < 1 && p->rows > 0) || (p->y_div && p->y_rows < 1 && p->rows > 0))
    return fail_status(SITU_E_BAD_SHAPE, "x_rows %d, y_rows %d", p->x_rows, p->y_rows);
  const int out_size = p->out_dtype == SITU_OUT_F32 ? 4 : 2;
  const int32_t n = p->n, k = p->k;
  if (p->rows > 0) {
    st = mode == situ::kGDgrad ? check_out("x", p->x, p->x_stride, k, out_size) : check_in("x", p->x, p->x_stride, k, 2);
    if (st != SITU_OK) return st;
    st = fwd ? check_out("y", p->y, p->y_stride, n, out_size) : check_in("y", p->y, p->y_stride, n, 2);
    if (st != SITU_OK) return st;
  } else if (!wgrad) {
    nothing = true;
    return SITU_OK;
  }
  st = wgrad ? check_out("w", p->w, k, k, out_size) : check_in("w", p->w, k, k, 2);
  if (st != SITU_OK) return st;

  a = situ::GroupedArgs{};
  a.offsets = p->offsets;
  a.pairs = indexed ? p->pairs : nullptr;
  a.rows = p->rows;
  a.experts = p->experts;
  a.out_f32 = p->out_dtype == SITU_OUT_F32;
  const situ::RowDiv xd = situ::make_row_div(p->x_div), yd = situ::make_row_div(p->y_div);
  const int32_t x_rows = p->x_div ? p->x_rows : p->rows, y_rows = p->y_div ? p->y_rows : p->rows;
  int64_t out_stride;
  if (fwd) {
    a.t = static_cast<const uint8_t*>(p->x); a.t_stride = 2 * p->x_stride; a.t_div = xd; a.t_rows = x_rows;
    a.c = static_cast<const uint8_t*>(p->w); a.c_stride = 2 * (int64_t)k; a.c_expert = 2 * (int64_t)n * k;
    a.out = p->y; out_stride = p->y_stride; a.o_div = yd; a.o_rows = y_rows;
    a.N = n; a.K = k;
  } else if (mode == situ::kGDgrad) {
    a.t = static_cast<const uint8_t*>(p->y); a.t_stride = 2 * p->y_stride; a.t_div = yd; a.t_rows = y_rows;
    a.c = static_cast<const uint8_t*>(p->w); a.c_stride = 2 * (int64_t)k; a.c_expert = 2 * (int64_t)n * k;
    a.out = p->x; out_stride = p->x_stride; a.o_div = xd; a.o_rows = x_rows;
    a.N = k; a.K = n;
  } else {
    a.t = static_cast<const uint8_t*>(p->y); a.t_stride = 2 * p->y_stride; a.t_div = yd; a.t_rows = y_rows;
    a.c = static_cast<const uint8_t*>(p->x); a.c_stride = 2 * p->x_stride; a.c_div = xd; a.c_rows = x_rows;
    a.out = p->w; out_stride = k; a.out_expert = (int64_t)n * k * out_size;
    a.M = n; a.N = k; a.K = p->rows;
  }
  a.out_stride = out_stride * out_size;
  a.vec = aligned(a.out, 16) && a.out_stride % 16 == 0;
  return SITU_OK;
}

situ_status fp8_args(const situ_moe_fp8_matmul_t* p, situ::GroupedArgs& a, bool& nothing) {
  nothing = false;
  if (!p) return fail_status(SITU_E_NULL_ARG, "args is NULL");
  situ_status st = check_sizes(p->rows, p->n, p->k, p->experts, p->out_dtype, p->reserved, p->offsets);
  if (st != SITU_OK) return st;
  if (p->k % 16) return fail_status(SITU_E_BAD_SHAPE, "k %d must be a multiple of 16", p->k);
  if ((nothing = p->rows == 0)) return SITU_OK;
  const int out_size = p->out_dtype == SITU_OUT_F32 ? 4 : 2;
  const int32_t kb = (p->k + 127) / 128;
  if ((st = check_in("a", p->a, p->a_stride, p->k, 1)) != SITU_OK) return st;
  if ((st = check_in("w", p->w, p->k, p->k, 1)) != SITU_OK) return st;
  if ((st = check_out("out", p->out, p->out_stride, p->n, out_size)) != SITU_OK) return st;
  if ((st = check_out("a_scale", p->a_scale, p->a_scale_stride, kb, 4)) != SITU_OK) return st;
  if (p->a_scale_stride >= kMaxScaleStride)
    return fail_status(SITU_E_UNSUPPORTED, "a_scale: stride %lld (below 2^22)", (long long)p->a_scale_stride);
  if ((st = check_out("w_scale", p->w_scale, kb, kb, 4)) != SITU_OK) return st;
  a = situ::GroupedArgs{};
  a.t = p->a; a.t_stride = p->a_stride; a.t_rows = p->rows;
  a.c = p->w; a.c_stride = p->k; a.c_expert = (int64_t)p->n * p->k;
  a.t_scale = p->a_scale; a.ts_stride = p->a_scale_stride; a.c_scale = p->w_scale;
  a.offsets = p->offsets;
  a.o_rows = p->rows;
  a.rows = p->rows; a.experts = p->experts;
  a.N = p->n; a.K = p->k;
  a.out = p->out; a.out_stride = p->out_stride * out_size; a.out_f32 = p->out_dtype == SITU_OUT_F32;
  a.vec = aligned(a.out, 16) && a.out_stride % 16 == 0;
  return SITU_OK;
}

// One launch of the call described by `a`.
situ_status launch(situ_status checked, bool nothing, situ::GroupedMode mode, situ::GroupedArgs& a, void* hip_stream,
                   const char* what) {
  if (checked != SITU_OK || nothing) return checked;
  int cus = 0;
  const situ_status st = situ::require_device(&cus);
  if (st != SITU_OK) return st;
  return launched(situ::launch_grouped(mode, a, cus, static_cast<hipStream_t>(hip_stream)), what);
}
const char* kernel(situ_status checked, bool nothing, situ::GroupedMode mode, const situ::GroupedArgs& a, int32_t cus) {
  if (checked != SITU_OK) return nullptr;
  if (nothing || cus < 1) {
    fail_status(SITU_E_BAD_SHAPE, nothing ? "a call without rows launches nothing" : "cus %d", cus);
    return nullptr;
  }
  return situ::grouped_kernel_name(mode, a, cus);
}

situ_status grouped(situ::GroupedMode mode, const situ_moe_grouped_t* p, void* hip_stream) {
  situ::GroupedArgs a;
  bool nothing;
  const situ_status st = grouped_args(mode, p, a, nothing);
  return launch(st, nothing, mode, a, hip_stream, "grouped matmul");
}

}  // namespace

extern "C" {

situ_status situ_moe_quantize_fp8_block128(const uint16_t* x, int64_t rows, int32_t cols, int64_t x_stride,
                                           uint8_t* codes, float* scales, void* hip_stream) {
  if (rows < 0 || cols <= 0 || cols % 16)
    return fail_status(SITU_E_BAD_SHAPE, "rows %lld, cols %d (a multiple of 16)", (long long)rows, cols);
  if (rows > kMaxRows || cols > kMaxSide)
    return fail_status(SITU_E_UNSUPPORTED, "rows %lld (at most 2^24), cols %d (2^18)", (long long)rows, cols);
  if (rows == 0) return SITU_OK;
  situ_status st = check_in("x", x, x_stride, cols, 2);
  if (st != SITU_OK) return st;
  if (!codes || !scales) return fail_status(SITU_E_NULL_ARG, "codes or scales is NULL");
  if (!aligned(codes, 8) || !aligned(scales, 4))
    return fail_status(SITU_E_BAD_SHAPE, "codes must be 8-byte and scales 4-byte aligned");
  int cus = 0;
  if ((st = situ::require_device(&cus)) != SITU_OK) return st;
  const situ::QuantBlockArgs q{x, x_stride, codes, scales, rows, cols};
  return launched(situ::launch_quant_block128(q, static_cast<hipStream_t>(hip_stream)), "quantize");
}

situ_status situ_moe_matmul_fp8_block128(const situ_moe_fp8_matmul_t* p, void* hip_stream) {
  situ::GroupedArgs a;
  bool nothing;
  const situ_status st = fp8_args(p, a, nothing);
  return launch(st, nothing, situ::kGFwd8, a, hip_stream, "FP8 matmul");
}

situ_status situ_moe_grouped_matmul(const situ_moe_grouped_t* args, void* hip_stream) {
  return grouped(situ::kGFwd, args, hip_stream);
}
situ_status situ_moe_grouped_matmul_dgrad(const situ_moe_grouped_t* args, void* hip_stream) {
  return grouped(situ::kGDgrad, args, hip_stream);
}
situ_status situ_moe_grouped_matmul_wgrad(const situ_moe_grouped_t* args, void* hip_stream) {
  return grouped(situ::kGWgrad, args, hip_stream);
}

const char* situ_moe_matmul_fp8_block128_kernel(const situ_moe_fp8_matmul_t* p, int32_t cus) {
  situ::GroupedArgs a;
  bool nothing;
  const situ_status st = fp8_args(p, a, nothing);
  return kernel(st, nothing, situ::kGFwd8, a, cus);
}
const char* situ_moe_grouped_matmul_kernel(int32_t direction, const situ_moe_grouped_t* p, int32_t cus) {
  constexpr situ::GroupedMode kModes[] = {situ::kGFwd, situ::kGDgrad, situ::kGWgrad};
  if (direction < 0 || direction > 2) {
    fail_status(SITU_E_UNSUPPORTED, "direction %d (0 the product, 1 dgrad, 2 wgrad)", direction);
    return nullptr;
  }
  situ::GroupedArgs a;
  bool nothing;
  const situ_status st = grouped_args(kModes[direction], p, a, nothing);
  return kernel(st, nothing, kModes[direction], a, cus);
}

}  // extern "C"
