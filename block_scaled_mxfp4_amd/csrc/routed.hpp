// Arguments and launchers of the steps around the routed products: the gate
// (router.hip), the gated activation (activation.hip), the combine
// (pair_combine.hip) and the adapters beside a projection (adapters.hip).
// routed_api.cpp checks what a caller passes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/situ_moe.h"

namespace situ {

// ---- the gate
// Workspace: [blocks][experts] partial probability sums, then as many partial
// counts, then the finishing kernel's ticket; none where one workgroup does it all.
constexpr int kRouterMaxExperts = 1024, kRouterMaxK = 64;
int router_blocks(int32_t tokens);
inline uint64_t router_workspace_bytes(int32_t tokens, int32_t experts) {
  const uint64_t blocks = (uint64_t)router_blocks(tokens);
  return blocks == 1 ? 0 : 8ull * blocks * (uint64_t)experts + 16;
}
hipError_t launch_router(const situ_moe_router_t& a, hipStream_t s);
hipError_t launch_router_backward(const situ_moe_router_backward_t& a, hipStream_t s);

// ---- the activation
hipError_t launch_activation(const situ_moe_activation_t& a, int cus, hipStream_t s);
hipError_t launch_activation_backward(const situ_moe_activation_t& a, int cus, hipStream_t s);

// ---- the combine
hipError_t launch_pair_combine(const situ_moe_combine_t& a, hipStream_t s);
hipError_t launch_pair_combine_backward(const situ_moe_combine_t& a, hipStream_t s);

// ---- the adapters
// Workspace: t, two bf16 terms or fp32 a row and rank; none where one launch does it all.
uint64_t adapters_workspace_bytes(const situ_moe_adapters_t& a);
hipError_t launch_adapters(const situ_moe_adapters_t& a, hipStream_t s);

}  // namespace situ
