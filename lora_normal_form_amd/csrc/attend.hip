// Attention of new tokens over the paged cache (scute_paged_attention,
// scute_sink_attention), and the host side of its forms.

#include "attend.h"

#include <algorithm>
#include <atomic>

#include "attend_host.h"

namespace scute {

void att_plain(const AttArgs& A, int es, int dp, int blocks, hipStream_t s) { att_form<ATT_PLAIN>(A, es, dp, blocks, s); }

int device_units(int device) {
  static std::atomic<int> known[64];
  const bool keep = device >= 0 && device < 64;
  int n = keep ? known[device].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, device) != hipSuccess || n < 1) return -1;
    if (keep) known[device].store(n, std::memory_order_relaxed);
  }
  return n;
}

int att_dim(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }
int64_t att_places(int units) { return (int64_t)units * ATT_PLACES; }
// the counters, and behind them the plan of calls over shared positions: the same
// place for heads of any size, so that nothing else is written to either
int64_t att_plan_place(int units) { return (4 * (ATT_ARRIVALS + 2 * att_places(units)) + 255) / 256 * 256; }
int64_t att_counter_bytes(int units) { return att_plan_place(units) + ATT_PLAN_BYTES; }
int64_t att_workspace(int units, int head_dim) {
  return att_counter_bytes(units) + att_places(units) * ATT_COLS * (att_dim(head_dim) + 4) * 4;
}

scute_status att_check(const char* fn, const AttCall& c) {
  const auto bad = [&](scute_status code, const char* what) { return fail(code, std::string(fn) + ": " + what); };
  const scute_kv_cache* C = c.C;
  scute_status st = check_cache(C, fn);
  if (st != SCUTE_OK) return st;
  if (c.n_heads < 1 || c.n_heads > 65536 || c.n_heads % C->n_kv_heads)
    return bad(SCUTE_E_SHAPE, "n_heads must be a multiple of n_kv_heads in [1, 65536]");
  if (c.n_requests < 0 || c.n_rows < 0 || c.n_rows > (1 << 20) || (!c.req && c.n_rows > c.n_requests))
    return bad(SCUTE_E_SHAPE, "n_rows must be in [0, 2^20], and without req at most n_requests");
  if (c.table_width < 1 || c.table_width > (1 << 24) || c.table_stride < c.table_width ||
      c.table_stride > ((int64_t)1 << 40))
    return bad(SCUTE_E_SHAPE, "table_width must be in [1, 2^24] and at most table_stride");
  if (c.window < 0) return bad(SCUTE_E_SHAPE, "window must be >= 0");
  if (c.sinks < 0) return bad(SCUTE_E_SHAPE, "sinks must be >= 0");
  // (the softmax runs on powers of two)
  if (!isfinite(c.scale * 1.4426950408889634f))
    return bad(SCUTE_E_INVALID, "scale, and scale log2(e) in fp32, must be finite");
  const int64_t wide = (int64_t)c.n_heads * C->head_dim, big = (int64_t)1 << 40;
  if (c.q_stride < 0 || c.q_stride > big || c.q_stride % 8 || c.out_stride < 0 || c.out_stride > big || c.out_stride % 8)
    return bad(SCUTE_E_SHAPE, "q_stride and out_stride must be multiples of 8 in [0, 2^40]");
  if (c.n_rows > 1 && c.out_stride < wide) return bad(SCUTE_E_SHAPE, "rows of out overlap");
  if (c.n_rows == 0) return SCUTE_OK;
  if (!c.q || (!c.table && c.n_requests) || !c.len || !c.out || !c.workspace)
    return bad(SCUTE_E_INVALID, "null pointer");
  if (((uintptr_t)c.q | (uintptr_t)c.out) & 15) return bad(SCUTE_E_INVALID, "q and out must be 16-byte aligned");
  if (((uintptr_t)c.table | (uintptr_t)c.len | (uintptr_t)c.req) & 3) return bad(SCUTE_E_INVALID, "misaligned pointer");
  if ((uintptr_t)c.workspace & 255) return bad(SCUTE_E_INVALID, "workspace must be 256-byte aligned");
  const int64_t es = C->dtype == SCUTE_F32 ? 4 : 2;
  if (c.q == c.out || rows_meet(c.q, c.q_stride * es, wide * es, c.out, c.out_stride * es, wide * es, c.n_rows))
    return bad(SCUTE_E_INVALID, "out is also q");
  return SCUTE_OK;
}

scute_status att_run(const char* fn, const AttCall& c, int form, hipStream_t s) {
  const scute_kv_cache* C = c.C;
  const int units = device_units(C->device), dp = att_dim(C->head_dim);
  if (units < 0) return fail(SCUTE_E_INVALID, std::string(fn) + ": no such HIP device");
  const int64_t counters = att_counter_bytes(units), need = att_workspace(units, C->head_dim);
  if (c.workspace_bytes < need) return fail(SCUTE_E_INVALID, std::string(fn) + ": the workspace is too small");
  const int64_t es = C->dtype == SCUTE_F32 ? 4 : 2;
  // t / page_size for 0 <= t < 2^31: multiply by ceil(2^(31 + shift) / page_size), shift = ceil(log2 page_size)
  int shift = 0;
  while ((1 << shift) < C->page_size) ++shift;
  const uint64_t mul = (((uint64_t)1 << (31 + shift)) + C->page_size - 1) / C->page_size;
  const int group = c.n_heads / C->n_kv_heads;
  const int64_t reach = std::min<int64_t>((int64_t)c.table_width * C->page_size, (int64_t)1 << 29);
  const int64_t unit = es == 4 ? 64 : 128;
  const int columns = group > 16 && att_widens((int)es, dp) ? 32 : 16;  // (of a query tile: att_mode)
  const int together = c.req && group <= 8 ? std::min(4, 16 / group) : 1;
  AttArgs A{c.q, C->k, C->v, c.out, c.table, c.len, c.req, (float*)((char*)c.workspace + counters), (int32_t*)c.workspace,
            c.q_stride, c.out_stride, C->page_stride, C->token_stride, C->head_stride, c.table_stride, C->n_pages, 0,
            (uint32_t)(need - counters), (uint32_t)mul, c.n_rows, C->n_kv_heads,
            (group + columns - 1) / columns, group, together, C->head_dim, C->page_size, shift, (int32_t)reach,
            c.n_requests, c.window, c.scale * 1.4426950408889634f, c.sinks};
  // rows of one launch: their units, at the table's whole width, stay below 2^31
  // (sinks: one tile more)
  const int64_t most = (((int64_t)1 << 31) - 1) /
                       ((int64_t)A.n_kv * A.q_tiles * (reach / unit + 2 + (form == ATT_SINKS) + ATT_EXTRA));
  if (most < 1) return fail(SCUTE_E_SHAPE, std::string(fn) + ": too many heads for a table this wide");
  for (int64_t r = 0; r < c.n_rows; r += most) {
    A.row0 = (int32_t)r;
    A.n_rows = (int32_t)std::min<int64_t>(most, c.n_rows - r);
    A.q = (const char*)c.q + r * c.q_stride * es;
    A.out = (char*)c.out + r * c.out_stride * es;
    A.len = c.len + r;
    A.req = c.req ? c.req + r : nullptr;
    (form == ATT_PLAIN ? att_plain : att_sinks)(A, (int)es, dp, units, s);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SCUTE_OK : hip_fail(e, fn);
}

}  // namespace scute

using namespace scute;

extern "C" scute_status scute_paged_attention_workspace(int32_t device, int32_t head_dim, int64_t* bytes) {
  if (!bytes) return fail(SCUTE_E_INVALID, "scute_paged_attention_workspace: bytes is null");
  if (device < 0) return fail(SCUTE_E_INVALID, "scute_paged_attention_workspace: device must be >= 0");
  if (head_dim < 8 || head_dim > 256 || head_dim % 8)
    return fail(SCUTE_E_SHAPE, "scute_paged_attention_workspace: head_dim must be a multiple of 8 in [8, 256]");
  const int units = device_units(device);
  if (units < 0) return fail(SCUTE_E_INVALID, "scute_paged_attention_workspace: no such HIP device");
  *bytes = att_workspace(units, head_dim);
  return SCUTE_OK;
}

namespace {

scute_status attention(const char* fn, const AttCall& c, int form, void* stream) {
  const scute_status st = att_check(fn, c);
  if (st != SCUTE_OK || c.n_rows == 0) return st;
  OnDevice g(c.C->device);
  if (!g.ok()) return hip_fail(g.err, fn);
  return att_run(fn, c, form, (hipStream_t)stream);
}

}  // namespace

extern "C" scute_status scute_paged_attention(const scute_kv_cache* C, const void* q, int64_t q_stride,
                                              int32_t n_heads, const int32_t* table, int64_t table_stride,
                                              int32_t n_requests, int32_t table_width, const int32_t* len,
                                              const int32_t* req, int32_t n_rows, float scale, int32_t window,
                                              void* out, int64_t out_stride, void* workspace,
                                              int64_t workspace_bytes, void* stream) {
  return attention("scute_paged_attention",
                   AttCall{C, q, q_stride, n_heads, table, table_stride, n_requests, table_width, len, req, n_rows, scale,
                           window, 0, out, out_stride, workspace, workspace_bytes},
                   ATT_PLAIN, stream);
}

extern "C" scute_status scute_sink_attention(const scute_kv_cache* C, const void* q, int64_t q_stride,
                                             int32_t n_heads, const int32_t* table, int64_t table_stride,
                                             int32_t n_requests, int32_t table_width, const int32_t* len,
                                             const int32_t* req, int32_t n_rows, float scale, int32_t window,
                                             int32_t sinks, void* out, int64_t out_stride, void* workspace,
                                             int64_t workspace_bytes, void* stream) {
  // (without a window every position is seen already)
  return attention("scute_sink_attention",
                   AttCall{C, q, q_stride, n_heads, table, table_stride, n_requests, table_width, len, req, n_rows, scale,
                           window, sinks, out, out_stride, workspace, workspace_bytes},
                   window > 0 && sinks > 0 ? ATT_SINKS : ATT_PLAIN, stream);
}
