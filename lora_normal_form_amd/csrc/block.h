// Shared by the operators between the adapter layers (block.hip, attend.hip).
#pragma once

#include "internal.h"

namespace scute {

// the cache's fields against their documented ranges; `fn` names the caller
scute_status check_cache(const scute_kv_cache* cache, const char* fn);

}  // namespace scute
