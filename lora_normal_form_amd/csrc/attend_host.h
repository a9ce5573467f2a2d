// The host side of attention over the paged cache (attend.hip), for its forms.
#pragma once

#include "block.h"

namespace scute {

struct AttArgs;

// Arguments of a call, as of scute_paged_attention, and sinks where it has them.
struct AttCall {
  const scute_kv_cache* C;
  const void* q;
  int64_t q_stride;
  int32_t n_heads;
  const int32_t* table;
  int64_t table_stride;
  int32_t n_requests, table_width;
  const int32_t *len, *req;
  int32_t n_rows;
  float scale;
  int32_t window, sinks;
  void* out;
  int64_t out_stride;
  void* workspace;
  int64_t workspace_bytes;
};
// the checks of a call's arguments (not the workspace's size); nothing touches the device
scute_status att_check(const char* fn, const AttCall& c);
// its launches, with the cache's device current
scute_status att_run(const char* fn, const AttCall& c, int form, hipStream_t s);

// compute units of `device`, asked once a device (a negative answer is an error)
int device_units(int device);
int att_dim(int head_dim);
int64_t att_workspace(int units, int head_dim);
constexpr int64_t ATT_PLAN_BYTES = 256;
int64_t att_plan_place(int units);

void att_plain(const AttArgs& A, int es, int dp, int blocks, hipStream_t s);
void att_sinks(const AttArgs& A, int es, int dp, int blocks, hipStream_t s);

}  // namespace scute
