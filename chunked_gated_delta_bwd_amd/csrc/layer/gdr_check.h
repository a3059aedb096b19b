// Checks of arguments that the operators around the delta rule share (host code).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../gdr_internal.h"

namespace gdr {
namespace check {

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline gdr_status hip_status(int err, const char* what) {
  if (err == 0) return GDR_OK;
  return set_error(GDR_EHIP, "%s: %s", what, hip_error_string(err));
}

struct Arg {
  const void* ptr;
  const char* name;
  bool required;
};

inline gdr_status check_ptrs(const Arg* a, int n) {
  for (int i = 0; i < n; ++i) {
    if (!a[i].ptr && a[i].required) return set_error(GDR_EINVAL, "%s is NULL", a[i].name);
    if (!aligned16(a[i].ptr)) return set_error(GDR_EINVAL, "%s is not 16-byte aligned", a[i].name);
  }
  return GDR_OK;
}

inline gdr_status check_ws(size_t need, const void* ws, size_t ws_bytes) {
  if (ws_bytes < need) return set_error(GDR_EWORKSPACE, "workspace %zu bytes, need %zu", ws_bytes, need);
  if (!ws && need) return set_error(GDR_EINVAL, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return set_error(GDR_EINVAL, "workspace is not 256-byte aligned");
  return GDR_OK;
}

// State pool and row slots of the single-token steps.
inline gdr_status check_pool(int32_t N, const float* state, int32_t P, const int32_t* slots) {
  if (P < 0) return set_error(GDR_EINVAL, "P (%d) must be >= 0", P);
  if (!slots && P < N) return set_error(GDR_EINVAL, "%d rows need as many states without slots (P = %d)", N, P);
  const Arg a[] = {{state, "state", P > 0}};
  gdr_status st = check_ptrs(a, 1);
  if (st != GDR_OK) return st;
  if (reinterpret_cast<uintptr_t>(slots) & 3u) return set_error(GDR_EINVAL, "slots is not 4-byte aligned");
  return GDR_OK;
}

}  // namespace check
}  // namespace gdr
