// Attention over the paged cache, of what rows have beside their shared positions.

#include "attend.h"
#include "attend_host.h"

namespace scute {

void att_suffix(const AttArgs& A, int es, int dp, int blocks, hipStream_t s) { att_form<ATT_SUFFIX>(A, es, dp, blocks, s); }

}  // namespace scute
