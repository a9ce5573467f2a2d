// Attention of new tokens over the paged cache (scute_paged_attention).

#include <math.h>

#include "block.h"
#include "kernels.h"

namespace scute {

struct AttArgs {
  const void *q, *k, *v;
  void* out;
  const int32_t *table, *len, *req;
  int64_t q_stride, out_stride, page_stride, token_stride, head_stride, table_stride, n_pages;
  int32_t n_heads, group, head_dim, page_size, table_width, n_requests, window;
  float scale_log2;  // scale * log2(e): the softmax runs on powers of two
};

template <typename T>
__device__ __forceinline__ float att_ld(const T* p) {
  if constexpr (sizeof(T) == 4)
    return ldg(p);
  else
    return bf2f(ldg(p));
}

// One work-group per (row, query head), its four waves on every fourth
// position, a lane on dims lane, lane + 64, ...; running maximum and sum per
// wave, the four joined in LDS.
template <typename T>
__global__ __launch_bounds__(256) void k_paged_attention(AttArgs A) {
  __shared__ float sm[4], sl[4], so[4][256];
  const int row = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int rq = A.req ? A.req[row] : row, D = A.head_dim;
  const int64_t reach = (int64_t)A.table_width * A.page_size;
  int n = rq >= 0 && rq < A.n_requests ? A.len[row] : 0;
  n = (int)(n < reach ? n : reach);
  const int lo = A.window > 0 && n > A.window ? n - A.window : 0;
  const T* q = (const T*)A.q + row * A.q_stride + (int64_t)h * D;
  const int64_t head = (h / A.group) * A.head_stride;
  float qv[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  for (int i = 0; i < 4; ++i) qv[i] = lane + 64 * i < D ? att_ld(q + lane + 64 * i) : 0.f;
  for (int t = lo + w; t < n; t += 4) {
    const int at = t / A.page_size;
    const int page = A.table[rq * A.table_stride + at];
    if (page < 0 || page >= A.n_pages) continue;
    const int64_t off = page * A.page_stride + (t - at * A.page_size) * A.token_stride + head;
    float s = 0.f;
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i < D) s += qv[i] * att_ld((const T*)A.k + off + lane + 64 * i);
    s = wave_sum(s) * A.scale_log2;
    const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - ref), p = exp2f(s - ref);
    m = mn;
    l = l * f + p;
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i < D) o[i] = o[i] * f + p * att_ld((const T*)A.v + off + lane + 64 * i);
  }
  if (lane == 0) sm[w] = m, sl[w] = l;
  for (int i = 0; i < 4; ++i) so[w][lane + 64 * i] = o[i];
  __syncthreads();
  const float mx = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3])), ref = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f, acc = 0.f;
  for (int i = 0; i < 4; ++i) {
    const float f = exp2f(sm[i] - ref);
    sum += sl[i] * f;
    acc += so[i][threadIdx.x] * f;
  }
  if ((int)threadIdx.x < D) {
    const float r[1] = {sum == 0.f ? 0.f : acc / sum};
    T* out = (T*)A.out + row * A.out_stride + (int64_t)h * D + threadIdx.x;
    if constexpr (sizeof(T) == 4)
      *out = r[0];
    else
      *out = (T)pack_bf2(__float_as_uint(r[0]), 0);
  }
}

}  // namespace scute

using namespace scute;

extern "C" scute_status scute_paged_attention_workspace(int32_t device, int32_t head_dim, int64_t* bytes) {
  if (!bytes) return fail(SCUTE_E_INVALID, "scute_paged_attention_workspace: bytes is null");
  if (device < 0) return fail(SCUTE_E_INVALID, "scute_paged_attention_workspace: device must be >= 0");
  if (head_dim < 8 || head_dim > 256 || head_dim % 8)
    return fail(SCUTE_E_SHAPE, "scute_paged_attention_workspace: head_dim must be a multiple of 8 in [8, 256]");
  *bytes = 256;
  return SCUTE_OK;
}

extern "C" scute_status scute_paged_attention(const scute_kv_cache* C, const void* q, int64_t q_stride,
                                              int32_t n_heads, const int32_t* table, int64_t table_stride,
                                              int32_t n_requests, int32_t table_width, const int32_t* len,
                                              const int32_t* req, int32_t n_rows, float scale, int32_t window,
                                              void* out, int64_t out_stride, void* workspace,
                                              int64_t workspace_bytes, void* stream) {
  const char* fn = "scute_paged_attention";
  scute_status st = check_cache(C, fn);
  if (st != SCUTE_OK) return st;
  if (n_heads < 1 || n_heads > 65536 || n_heads % C->n_kv_heads)
    return fail(SCUTE_E_SHAPE, "scute_paged_attention: n_heads must be a multiple of n_kv_heads in [1, 65536]");
  if (n_requests < 0 || n_rows < 0 || n_rows > (1 << 20) || (!req && n_rows > n_requests))
    return fail(SCUTE_E_SHAPE, "scute_paged_attention: n_rows must be in [0, 2^20], and without req at most n_requests");
  if (table_width < 1 || table_width > (1 << 24) || table_stride < table_width || table_stride > ((int64_t)1 << 40))
    return fail(SCUTE_E_SHAPE,
                "scute_paged_attention: table_width must be in [1, 2^24] and at most table_stride");
  if (window < 0) return fail(SCUTE_E_SHAPE, "scute_paged_attention: window must be >= 0");
  if (!isfinite(scale)) return fail(SCUTE_E_INVALID, "scute_paged_attention: scale must be finite");
  const int64_t wide = (int64_t)n_heads * C->head_dim, big = (int64_t)1 << 40;
  if (q_stride < 0 || q_stride > big || q_stride % 8 || out_stride < 0 || out_stride > big || out_stride % 8)
    return fail(SCUTE_E_SHAPE, "scute_paged_attention: q_stride and out_stride must be multiples of 8 in [0, 2^40]");
  if (n_rows > 1 && out_stride < wide) return fail(SCUTE_E_SHAPE, "scute_paged_attention: rows of out overlap");
  if (n_rows == 0) return SCUTE_OK;
  if (!q || !table || !len || !out || !workspace) return fail(SCUTE_E_INVALID, "scute_paged_attention: null pointer");
  if (((uintptr_t)q | (uintptr_t)out) & 15)
    return fail(SCUTE_E_INVALID, "scute_paged_attention: q and out must be 16-byte aligned");
  if (((uintptr_t)table | (uintptr_t)len | (uintptr_t)req) & 3)
    return fail(SCUTE_E_INVALID, "scute_paged_attention: misaligned pointer");
  if ((uintptr_t)workspace & 255) return fail(SCUTE_E_INVALID, "scute_paged_attention: workspace must be 256-byte aligned");
  if (q == out) return fail(SCUTE_E_INVALID, "scute_paged_attention: out is also q");
  DeviceGuard g(C->device);
  if (!g.ok()) return hip_fail(g.err, fn);
  int64_t need = 0;
  if ((st = scute_paged_attention_workspace(C->device, C->head_dim, &need)) != SCUTE_OK) return st;
  if (workspace_bytes < need) return fail(SCUTE_E_INVALID, "scute_paged_attention: the workspace is too small");
  const AttArgs A{q, C->k, C->v, out, table, len, req, q_stride, out_stride, C->page_stride, C->token_stride,
                  C->head_stride, table_stride, C->n_pages, n_heads, n_heads / C->n_kv_heads, C->head_dim,
                  C->page_size, table_width, n_requests, window, scale * 1.4426950408889634f};
  const dim3 grid((unsigned)n_rows, (unsigned)n_heads);
  const hipStream_t s = (hipStream_t)stream;
  if (C->dtype == SCUTE_F32)
    hipLaunchKernelGGL(k_paged_attention<float>, grid, dim3(256), 0, s, A);
  else
    hipLaunchKernelGGL(k_paged_attention<uint16_t>, grid, dim3(256), 0, s, A);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SCUTE_OK : hip_fail(e, fn);
}
