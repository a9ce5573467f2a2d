// Attention over the paged cache, with first positions that stay visible: paged
// attention whose tiles are the sinks' and then the window's, as if they lay side by
// side, so that the work is cut over both and a row costs what it sees. 128 rows up
// to 32000, window 4096, 16 sinks: 328 us, 2.0 GB, 6.2 TB/s, which is what bounds it.

#include "attend.h"
#include "attend_host.h"

namespace scute {

void att_sinks(const AttArgs& A, int es, int dp, int blocks, hipStream_t s) { att_form<ATT_SINKS>(A, es, dp, blocks, s); }

}  // namespace scute
