// What the entry points beside the layer check of a caller's arguments (host).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.hpp"

namespace situ {

constexpr int64_t kMaxStride = (int64_t)1 << 40;

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline situ_status launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return SITU_OK;
  return fail_status(SITU_E_LAUNCH, "%s launch failed: %s", what, hipGetErrorString(e));
}

// Rows of `width` elements of `size` bytes that are read and written 16 bytes at a time.
inline situ_status check_in(const char* name, const void* p, int64_t stride, int32_t width, int size) {
  if (!p) return fail_status(SITU_E_NULL_ARG, "%s is NULL", name);
  if (!aligned(p, 16)) return fail_status(SITU_E_BAD_SHAPE, "%s must be 16-byte aligned", name);
  if (stride < width || stride > kMaxStride || stride * size % 16)
    return fail_status(SITU_E_BAD_SHAPE, "%s: stride %lld (at least %d, a multiple of %d)", name, (long long)stride,
                       width, 16 / size);
  return SITU_OK;
}
// Rows without such a demand.
inline situ_status check_out(const char* name, const void* p, int64_t stride, int32_t width, int size) {
  if (!p) return fail_status(SITU_E_NULL_ARG, "%s is NULL", name);
  if (!aligned(p, (uintptr_t)size)) return fail_status(SITU_E_BAD_SHAPE, "%s must be %d-byte aligned", name, size);
  if (stride < width || stride > kMaxStride)
    return fail_status(SITU_E_BAD_SHAPE, "%s: stride %lld (at least %d)", name, (long long)stride, width);
  return SITU_OK;
}
// A dense array.
inline situ_status check_array(const char* name, const void* p, uintptr_t align) {
  if (!p) return fail_status(SITU_E_NULL_ARG, "%s is NULL", name);
  if (!aligned(p, align)) return fail_status(SITU_E_BAD_SHAPE, "%s must be %d-byte aligned", name, (int)align);
  return SITU_OK;
}

}  // namespace situ
