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

// the cache's fields against their documented ranges; `fn` names the caller
scute_status check_cache(const scute_kv_cache* cache, const char* fn);

}  // namespace scute
