// Shared by the operators between the adapter layers (block.hip, attend.hip).
#pragma once

#include "internal.h"

namespace scute {

// Runs with `dev` current and restores the caller's device afterwards; ok() is
// false if `dev` cannot be made current.
struct OnDevice {
  int prev = -1;
  bool active = false;
  hipError_t err;
  explicit OnDevice(int dev) {
    if ((err = hipGetDevice(&prev)) != hipSuccess || prev == dev) return;
    err = hipSetDevice(dev);
    active = err == hipSuccess;
  }
  ~OnDevice() {
    if (active) (void)hipSetDevice(prev);
  }
  bool ok() const { return err == hipSuccess; }
};

// Whether rows of `wide` bytes at `a` and `b` (n each, sa and sb bytes apart)
// are seen to share a byte. Column ranges of one buffer do not; of rows with
// different strides it is said only where their extents are one row each.
inline bool rows_meet(const void* a, int64_t sa, int64_t wa, const void* b, int64_t sb, int64_t wb, int64_t n) {
  if (!a || !b || n < 1) return false;
  const int64_t d = (int64_t)((uintptr_t)b - (uintptr_t)a);
  if (n == 1) return d < wa && -d < wb;
  if (sa != sb || sa <= 0) return false;
  // row j of b begins `off` bytes into the place of row j + k of a
  const int64_t k = d >= 0 ? d / sa : -((-d + sa - 1) / sa), off = d - k * sa;
  return (k < n && -k < n && off < wa) || (k + 1 < n && -(k + 1) < n && off + wb > sa);
}

// the cache's fields against their documented ranges; `fn` names the caller
scute_status check_cache(const scute_kv_cache* cache, const char* fn);

}  // namespace scute
