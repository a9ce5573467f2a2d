// Attention over the paged cache, with first positions that stay visible.

#include "attend.h"
#include "attend_host.h"

namespace scute {

void att_sinks(const AttArgs& A, int es, int dp, int blocks, hipStream_t s) { att_form<ATT_SINKS>(A, es, dp, blocks, s); }

}  // namespace scute
