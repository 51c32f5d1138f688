// Entry points of the steps around the routed products: argument checks, then
// the launches.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/situ_moe.h"
#include "checks.hpp"
#include "internal.hpp"
#include "routed.hpp"

namespace {

using situ::aligned;
using situ::check_array;
using situ::check_in;
using situ::check_out;
using situ::fail_status;
using situ::launched;

constexpr int32_t kMaxRows = 1 << 24, kMaxSide = 1 << 18, kMaxInner = 1 << 17, kMaxExperts = 1024, kMaxSlots = 1024;
constexpr int32_t kMaxRank = 256, kMaxRequests = 1 << 20;

int size_of(int32_t dtype) { return dtype == SITU_OUT_F32 ? 4 : 2; }

situ_status check_dtype(const char* name, int32_t dtype) {
  if (dtype == SITU_OUT_F32 || dtype == SITU_OUT_BF16) return SITU_OK;
  return fail_status(SITU_E_UNSUPPORTED, "%s %d", name, dtype);
}
situ_status check_flag(const char* name, int32_t v) {
  if (v == 0 || v == 1) return SITU_OK;
  return fail_status(SITU_E_BAD_SHAPE, "%s is %d, not 0 or 1", name, v);
}

#define SITU_TRY(e)                        \
  do {                                     \
    const situ_status try_st = (e);        \
    if (try_st != SITU_OK) return try_st;  \
  } while (0)

// What the gate and its gradient share.
situ_status check_gate(int32_t tokens, int32_t experts, int32_t top_k, int32_t scoring, int32_t logits_dtype,
                       int32_t renormalize, float scale) {
  if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts)
    return fail_status(SITU_E_BAD_SHAPE, "tokens %d, experts %d, top_k %d", tokens, experts, top_k);
  if (tokens > kMaxRows || experts > situ::kRouterMaxExperts || top_k > situ::kRouterMaxK)
    return fail_status(SITU_E_UNSUPPORTED, "tokens %d (at most 2^24), experts %d (1024), top_k %d (64)", tokens, experts,
                       top_k);
  if (scoring != SITU_SCORE_SOFTMAX && scoring != SITU_SCORE_SIGMOID)
    return fail_status(SITU_E_UNSUPPORTED, "scoring %d", scoring);
  SITU_TRY(check_dtype("logits_dtype", logits_dtype));
  SITU_TRY(check_flag("renormalize", renormalize));
  if (!(fabsf(scale) < INFINITY)) return fail_status(SITU_E_BAD_SHAPE, "scale is not finite");
  return SITU_OK;
}

situ_status check_router(const situ_moe_router_t* p) {
  if (!p) return fail_status(SITU_E_NULL_ARG, "args is NULL");
  SITU_TRY(check_gate(p->tokens, p->experts, p->top_k, p->scoring, p->logits_dtype, p->renormalize, p->scale));
  SITU_TRY(check_dtype("weights_dtype", p->weights_dtype));
  if (p->bias && p->scoring != SITU_SCORE_SIGMOID)
    return fail_status(SITU_E_UNSUPPORTED, "a bias needs sigmoid scores");
  const int given = (p->counts != nullptr) + (p->prob_sum != nullptr) + (p->loss != nullptr);
  if (given != 0 && given != 3) return fail_status(SITU_E_NULL_ARG, "counts, prob_sum and loss are given together or not at all");
  return SITU_OK;
}
uint64_t router_bytes(const situ_moe_router_t* p) {
  return p->counts ? situ::router_workspace_bytes(p->tokens, p->experts) : 0;
}

// What the activation and its gradient share.
situ_status check_activation(const situ_moe_activation_t* p) {
  if (!p) return fail_status(SITU_E_NULL_ARG, "args is NULL");
  if (p->rows < 0 || p->inner < 8 || p->inner % 8 || p->experts < 1)
    return fail_status(SITU_E_BAD_SHAPE, "rows %d, inner %d (a multiple of 8), experts %d", p->rows, p->inner, p->experts);
  if (p->rows > kMaxRows || p->inner > kMaxInner || p->experts > kMaxExperts)
    return fail_status(SITU_E_UNSUPPORTED, "rows %d (at most 2^24), inner %d (2^17), experts %d (1024)", p->rows, p->inner,
                       p->experts);
  if (p->activation < SITU_ACTIVATION_SITU || p->activation > SITU_ACTIVATION_SWIGLU_BIAS)
    return fail_status(SITU_E_UNSUPPORTED, "activation %d", p->activation);
  if (!p->offsets && p->experts != 1) return fail_status(SITU_E_NULL_ARG, "offsets is NULL with %d experts", p->experts);
  if (!aligned(p->offsets, 4)) return fail_status(SITU_E_BAD_SHAPE, "offsets must be 4-byte aligned");
  if (p->activation != SITU_ACTIVATION_SWIGLU) {
    const bool situ = p->activation == SITU_ACTIVATION_SITU;
    SITU_TRY(check_array(situ ? "situ_beta" : "swiglu_alpha", p->p0, 4));
    SITU_TRY(check_array(situ ? "situ_linear_beta" : "swiglu_beta", p->p1, 4));
  }
  if ((p->codes == nullptr) != (p->scales == nullptr))
    return fail_status(SITU_E_NULL_ARG, "codes and scales are given together or not at all");
  if (!aligned(p->codes, 8) || !aligned(p->scales, 4))
    return fail_status(SITU_E_BAD_SHAPE, "codes must be 8-byte and scales 4-byte aligned");
  return SITU_OK;
}

situ_status check_combine(const situ_moe_combine_t* p, bool backward) {
  if (!p) return fail_status(SITU_E_NULL_ARG, "args is NULL");
  if (p->tokens < 0 || p->rows < 0 || p->top_k < 1 || p->hidden < 8 || p->hidden % 8)
    return fail_status(SITU_E_BAD_SHAPE, "tokens %d, top_k %d, hidden %d (a multiple of 8), rows %d", p->tokens, p->top_k,
                       p->hidden, p->rows);
  if (p->tokens > kMaxRows || p->rows > kMaxRows || p->top_k > kMaxSlots || p->hidden > kMaxSide)
    return fail_status(SITU_E_UNSUPPORTED, "tokens %d, rows %d (at most 2^24), top_k %d (1024), hidden %d (2^18)", p->tokens,
                       p->rows, p->top_k, p->hidden);
  if (p->reserved != 0) return fail_status(SITU_E_BAD_SHAPE, "reserved is %d, not 0", p->reserved);
  SITU_TRY(check_dtype("y_dtype", p->y_dtype));
  SITU_TRY(check_dtype("weights_dtype", p->weights_dtype));
  SITU_TRY(check_dtype("out_dtype", p->out_dtype));
  if (p->tokens == 0) return SITU_OK;
  SITU_TRY(check_array("weights", p->weights, (uintptr_t)size_of(p->weights_dtype)));
  SITU_TRY(check_array("inv", p->inv, 4));
  SITU_TRY(check_in(backward ? "d_out" : "out", p->out, p->out_stride, p->hidden, size_of(p->out_dtype)));
  const bool reads_y = !backward || p->d_weights;
  if (p->rows > 0 && reads_y) SITU_TRY(check_in("y", p->y, p->y_stride, p->hidden, size_of(p->y_dtype)));
  if (backward) {
    if (!p->dy && !p->d_weights) return fail_status(SITU_E_NULL_ARG, "dy and d_weights are NULL");
    if (p->rows > 0 && p->dy) SITU_TRY(check_in("dy", p->dy, p->dy_stride, p->hidden, size_of(p->y_dtype)));
    if (!aligned(p->d_weights, 4)) return fail_status(SITU_E_BAD_SHAPE, "d_weights must be 4-byte aligned");
  }
  return SITU_OK;
}

situ_status check_adapter_sizes(const situ_moe_adapters_t* p) {
  if (!p) return fail_status(SITU_E_NULL_ARG, "args is NULL");
  if (p->rows < 0 || p->n < 8 || p->k < 8 || p->rank < 8 || p->n % 8 || p->k % 8 || p->rank % 8)
    return fail_status(SITU_E_BAD_SHAPE, "rows %d, n %d, k %d, rank %d (multiples of 8)", p->rows, p->n, p->k, p->rank);
  if (p->rows > kMaxRows || p->n > kMaxSide || p->k > kMaxSide || p->rank > kMaxRank)
    return fail_status(SITU_E_UNSUPPORTED, "rows %d (at most 2^24), n %d, k %d (2^18), rank %d (256)", p->rows, p->n, p->k,
                       p->rank);
  return SITU_OK;
}

situ_status check_workspace(const void* ws, uint64_t bytes, uint64_t need) {
  if (need == 0) return SITU_OK;
  if (!ws || bytes < need)
    return fail_status(SITU_E_WORKSPACE, "workspace of %llu bytes, %llu needed", ws ? (unsigned long long)bytes : 0ull,
                       (unsigned long long)need);
  if (!aligned(ws, 16)) return fail_status(SITU_E_BAD_SHAPE, "workspace must be 16-byte aligned");
  return SITU_OK;
}

hipStream_t stream(void* s) { return static_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

situ_status situ_moe_router_workspace(const situ_moe_router_t* p, uint64_t* bytes) {
  SITU_TRY(check_router(p));
  if (!bytes) return fail_status(SITU_E_NULL_ARG, "bytes is NULL");
  *bytes = router_bytes(p);
  return SITU_OK;
}

situ_status situ_moe_router(const situ_moe_router_t* p, void* hip_stream) {
  SITU_TRY(check_router(p));
  if (p->tokens == 0 && !p->counts) return SITU_OK;
  if (p->tokens > 0) {
    SITU_TRY(check_out("logits", p->logits, p->logits_stride, p->experts, size_of(p->logits_dtype)));
    SITU_TRY(check_array("ids", p->ids, 4));
    if (!aligned(p->weights, (uintptr_t)size_of(p->weights_dtype)) || !aligned(p->packed, 4) || !aligned(p->bias, 4))
      return fail_status(SITU_E_BAD_SHAPE, "weights, packed and bias must be aligned to their elements");
  }
  if (!aligned(p->counts, 4) || !aligned(p->prob_sum, 4) || !aligned(p->loss, 4))
    return fail_status(SITU_E_BAD_SHAPE, "counts, prob_sum and loss must be 4-byte aligned");
  SITU_TRY(check_workspace(p->workspace, p->workspace_bytes, router_bytes(p)));
  int cus = 0;
  SITU_TRY(situ::require_device(&cus));
  return launched(situ::launch_router(*p, stream(hip_stream)), "router");
}

situ_status situ_moe_router_backward(const situ_moe_router_backward_t* p, void* hip_stream) {
  if (!p) return fail_status(SITU_E_NULL_ARG, "args is NULL");
  SITU_TRY(check_gate(p->tokens, p->experts, p->top_k, p->scoring, p->logits_dtype, p->renormalize, p->scale));
  SITU_TRY(check_dtype("out_dtype", p->out_dtype));
  if ((p->counts == nullptr) != (p->d_loss == nullptr))
    return fail_status(SITU_E_NULL_ARG, "counts and d_loss are given together or not at all");
  if (p->tokens == 0) return SITU_OK;                // empty arrays may be NULL
  if (!p->counts && !p->d_weights) return fail_status(SITU_E_NULL_ARG, "neither d_weights nor d_loss is given");
  SITU_TRY(check_out("logits", p->logits, p->logits_stride, p->experts, size_of(p->logits_dtype)));
  SITU_TRY(check_out("d_logits", p->d_logits, p->out_stride, p->experts, size_of(p->out_dtype)));
  if (p->d_weights) SITU_TRY(check_array("ids", p->ids, 4));
  if (!aligned(p->d_weights, 4) || !aligned(p->counts, 4) || !aligned(p->d_loss, 4))
    return fail_status(SITU_E_BAD_SHAPE, "d_weights, counts and d_loss must be 4-byte aligned");
  int cus = 0;
  SITU_TRY(situ::require_device(&cus));
  return launched(situ::launch_router_backward(*p, stream(hip_stream)), "router backward");
}

situ_status situ_moe_activation(const situ_moe_activation_t* p, void* hip_stream) {
  SITU_TRY(check_activation(p));
  if (p->rows == 0) return SITU_OK;
  SITU_TRY(check_in("gate_up", p->gate_up, p->gate_up_stride, 2 * p->inner, 2));
  SITU_TRY(check_in("h", p->h, p->h_stride, p->inner, 2));
  int cus = 0;
  SITU_TRY(situ::require_device(&cus));
  return launched(situ::launch_activation(*p, cus, stream(hip_stream)), "activation");
}

situ_status situ_moe_activation_backward(const situ_moe_activation_t* p, void* hip_stream) {
  SITU_TRY(check_activation(p));
  if (p->rows == 0) return SITU_OK;
  if ((p->gate_up != nullptr) == (p->codes != nullptr))
    return fail_status(SITU_E_NULL_ARG, "either gate_up or codes and scales are given");
  if (p->gate_up) SITU_TRY(check_in("gate_up", p->gate_up, p->gate_up_stride, 2 * p->inner, 2));
  if (p->h) SITU_TRY(check_in("h", p->h, p->h_stride, p->inner, 2));
  SITU_TRY(check_in("dh", p->dh, p->dh_stride, p->inner, 2));
  SITU_TRY(check_in("d_gate_up", p->d_gate_up, p->d_gate_up_stride, 2 * p->inner, 2));
  int cus = 0;
  SITU_TRY(situ::require_device(&cus));
  return launched(situ::launch_activation_backward(*p, cus, stream(hip_stream)), "activation backward");
}

situ_status situ_moe_combine(const situ_moe_combine_t* p, void* hip_stream) {
  SITU_TRY(check_combine(p, false));
  if (p->tokens == 0) return SITU_OK;
  int cus = 0;
  SITU_TRY(situ::require_device(&cus));
  return launched(situ::launch_pair_combine(*p, stream(hip_stream)), "combine");
}

situ_status situ_moe_combine_backward(const situ_moe_combine_t* p, void* hip_stream) {
  SITU_TRY(check_combine(p, true));
  if (p->tokens == 0) return SITU_OK;
  int cus = 0;
  SITU_TRY(situ::require_device(&cus));
  return launched(situ::launch_pair_combine_backward(*p, stream(hip_stream)), "combine backward");
}

situ_status situ_moe_adapters_workspace(const situ_moe_adapters_t* p, uint64_t* bytes) {
  SITU_TRY(check_adapter_sizes(p));
  if (!bytes) return fail_status(SITU_E_NULL_ARG, "bytes is NULL");
  *bytes = situ::adapters_workspace_bytes(*p);
  return SITU_OK;
}

situ_status situ_moe_adapters(const situ_moe_adapters_t* p, void* hip_stream) {
  SITU_TRY(check_adapter_sizes(p));
  if (p->requests < 1 || p->adapters < 1)
    return fail_status(SITU_E_BAD_SHAPE, "requests %d, adapters %d", p->requests, p->adapters);
  if (p->requests > kMaxRequests || p->adapters > kMaxRequests)
    return fail_status(SITU_E_UNSUPPORTED, "requests %d, adapters %d (at most 2^20)", p->requests, p->adapters);
  SITU_TRY(check_dtype("out_dtype", p->out_dtype));
  if (p->reserved != 0) return fail_status(SITU_E_BAD_SHAPE, "reserved is %d, not 0", p->reserved);
  if (p->rows == 0) return SITU_OK;
  SITU_TRY(check_array("offsets", p->offsets, 4));
  SITU_TRY(check_array("adapter", p->adapter, 4));
  if (!aligned(p->ranks, 4) || !aligned(p->scales, 4))
    return fail_status(SITU_E_BAD_SHAPE, "ranks and scales must be 4-byte aligned");
  SITU_TRY(check_in("x", p->x, p->x_stride, p->k, 2));
  SITU_TRY(check_array("a", p->a, 16));
  SITU_TRY(check_array("b", p->b, 16));
  if (p->base) SITU_TRY(check_in("base", p->base, p->base_stride, p->n, size_of(p->out_dtype)));
  SITU_TRY(check_in("out", p->out, p->out_stride, p->n, size_of(p->out_dtype)));
  SITU_TRY(check_workspace(p->workspace, p->workspace_bytes, situ::adapters_workspace_bytes(*p)));
  int cus = 0;
  SITU_TRY(situ::require_device(&cus));
  return launched(situ::launch_adapters(*p, stream(hip_stream)), "adapters");
}

}  // extern "C"
