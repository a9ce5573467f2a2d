// Operators between a decoder block's adapter layers: pages and slots of a
// step's tokens (scute_cache_assign), rotary positions with the cache store
// (scute_rotary_store) and the norms around the residual
// (scute_residual_norm). The attention over the cache is in attend.hip.

#include <math.h>

#include <algorithm>

#include "block.h"
#include "kernels.h"

namespace scute {

// ---------------------------------------------------------------------------
// pages and slots from the requests' lengths
// ---------------------------------------------------------------------------

// Every work-group computes the same three exclusive prefix sums over the
// requests (tokens, pages wanted, pages returned), thread i over the
// contiguous requests [i per, (i + 1) per), and keeps only the sums at the
// threads' borders in LDS. A flat index (token, page taken, page returned) is
// then found by a binary search over the borders and a walk over at most
// `per` requests, so the whole step is one launch with no exchange between
// work-groups: redoing the sums (8 bytes a request from L2) costs less than a
// second launch. Bound by that chain of latencies, not by bytes (128 requests of
// one token: 5.7 us; 2000 requests of up to 150 tokens: 10.4 us; the work-groups'
// own sums grow with the requests: 65536 of one token 371 us). Sums saturate
// at 2^30 (saturating addition of non-negative numbers is associative, so a
// scan may use it).
constexpr int ASG_THREADS = 1024;
constexpr uint32_t ASG_MAX = 1u << 30;

// the call's arguments, and x / page_size = x mul >> 31 + shift for x < 2^31
struct AsgArgs {
  scute_cache_assign_args a;
  uint32_t mul, shift;
};

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;  // both at most 2^30
  return s < ASG_MAX ? s : ASG_MAX;
}

struct AsgReq {
  uint32_t old, add, rows;    // positions held, tokens brought, rows of them
  uint32_t held, want, gone;  // pages held, wanted, returned
  bool fits, ends;
};

__device__ __forceinline__ uint32_t asg_page(const AsgArgs& A, uint32_t x) {
  return (uint32_t)(((uint64_t)x * A.mul) >> (31 + A.shift));
}

// FLAGS: the call has some (128 requests 5.7 us, 2000 requests 10.4; with the
// tests for them in every call 5.9 and 10.7)
template <bool FLAGS>
__device__ __forceinline__ AsgReq asg_req(const AsgArgs& A, int32_t o, int32_t n) {
  AsgReq q;
  q.old = o > 0 ? min((uint32_t)o, ASG_MAX) : 0u;
  q.ends = n < 0;
  q.add = n > 0 ? min((uint32_t)n, ASG_MAX / 2) : 0u;
  const bool one_each = FLAGS && (A.a.flags & SCUTE_ASSIGN_ONE_EACH);
  q.rows = one_each ? 1u : q.add;
  const uint32_t ps = (uint32_t)A.a.page_size;
  q.held = asg_page(A, q.old + ps - 1);
  const uint32_t upto = asg_page(A, q.old + q.add + ps - 1);
  q.fits = !q.ends && upto <= (uint32_t)A.a.table_width && !(one_each && q.add > 1);
  q.want = q.fits ? upto - q.held : 0u;
  q.gone = q.ends ? min(q.held, (uint32_t)A.a.table_width) : 0u;
  return q;
}

// inclusive saturating sum over the wave's lanes (row shifts and broadcasts)
__device__ __forceinline__ uint32_t sat_scan(uint32_t v) {
#define STEP(ctrl, rows) v = sat_add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, false))
  STEP(0x111, 0xF);
  STEP(0x112, 0xF);
  STEP(0x114, 0xF);
  STEP(0x118, 0xF);
  STEP(0x142, 0xA);
  STEP(0x143, 0xC);
#undef STEP
  return v;
}

// index of the last border that is <= x (borders ascending, b[0] = 0)
__device__ __forceinline__ int asg_find(const uint32_t* b, uint32_t x) {
  int lo = 0;
#pragma unroll
  for (int step = ASG_THREADS / 2; step > 0; step >>= 1)
    if (b[lo + step] <= x) lo += step;
  return lo;
}

template <bool FLAGS>
__global__ __launch_bounds__(ASG_THREADS) void k_cache_assign(AsgArgs G) {
  const scute_cache_assign_args& A = G.a;
  __shared__ uint32_t ctok[ASG_THREADS], cpage[ASG_THREADS], cgone[ASG_THREADS];
  __shared__ int32_t s_old[ASG_THREADS], s_new[ASG_THREADS];  // lengths, up to a request a thread
  __shared__ uint32_t wsum[3][ASG_THREADS / 64], wout[3][ASG_THREADS / 64];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int R = A.n_requests, per = (R + ASG_THREADS - 1) / ASG_THREADS;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  const int64_t head = A.cursor[0], tail = A.cursor[1];

  uint32_t own[3] = {0, 0, 0};
  for (int r = r0; r < r1; ++r) {
    const int32_t o = A.old_len[r], n = A.new_len[r];
    const AsgReq q = asg_req<FLAGS>(G, o, n);
    own[0] = sat_add(own[0], q.rows);
    own[1] = sat_add(own[1], q.want);
    own[2] = sat_add(own[2], q.gone);
    if (per == 1) s_old[tid] = o, s_new[tid] = n;
  }
  uint32_t inc[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    inc[k] = sat_scan(own[k]);
    if (lane == 63) wsum[k][wv] = inc[k];
  }
  __syncthreads();
  uint32_t pre[3], tot[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < ASG_THREADS / 64; ++w) {
      before = w == wv ? all : before;
      all = sat_add(all, wsum[k][w]);
    }
    const uint32_t left = (uint32_t)__shfl_up((int)inc[k], 1, 64);
    pre[k] = sat_add(before, lane ? left : 0u);
    tot[k] = all;
  }
  ctok[tid] = pre[0];
  cpage[tid] = pre[1];
  cgone[tid] = pre[2];
  // whether the request's tokens, the first of them token `tok`, all have rows
  // (where one's have not, neither have those of any that follow: pages are
  // taken up to it, and the sums before it hold as they are)
  const auto has_rows = [&](const AsgReq& q, uint32_t tok) {
    return !FLAGS || !(A.flags & SCUTE_ASSIGN_FIT_ROWS) || q.add == 0 || tok + q.add <= (uint32_t)A.max_tokens;
  };
  const auto request = [&](int r) {
    return per == 1 ? asg_req<FLAGS>(G, s_old[r], s_new[r]) : asg_req<FLAGS>(G, A.old_len[r], A.new_len[r]);
  };

  const uint32_t cap = (uint32_t)A.ring_size;
  const int64_t free64 = tail - head;
  const uint32_t avail = free64 <= 0 ? 0u : free64 < (int64_t)cap ? (uint32_t)free64 : cap;
  const uint32_t h0 = (uint32_t)((uint64_t)head % cap), t0 = (uint32_t)((uint64_t)tail % cap);
  // pages taken: requests that want pages are placed up to the first that the
  // free pages do not cover
  uint32_t taken = 0;
  {
    uint32_t tok = pre[0], page = pre[1], placed = 0, refused = 0;
    for (int r = r0; r < r1; ++r) {
      const AsgReq q = request(r);
      const uint32_t need = sat_add(page, q.want);
      const bool ok = q.fits && (q.want == 0 || need <= avail) && has_rows(q, tok);
      if (ok && q.want) taken = need;
      if (ok) placed = sat_add(placed, q.add);
      refused += !q.ends && !ok;
      if (blockIdx.x == 0) {
        A.cu_len[r] = (int32_t)tok;
        A.seq_len[r] = q.ends ? 0 : (int32_t)(ok ? q.old + q.add : q.old);
      }
      tok = sat_add(tok, q.rows);
      page = need;
    }
    // (within a wave the last lane with pages taken has the most)
    const uint64_t some = __ballot(taken != 0);
    taken = some ? (uint32_t)__shfl((int)taken, 63 - __clzll((long long)some), 64) : 0u;
    if (blockIdx.x == 0) {
      for (int o = 32; o > 0; o >>= 1) {
        placed = sat_add(placed, (uint32_t)__shfl_xor((int)placed, o, 64));
        refused += (uint32_t)__shfl_xor((int)refused, o, 64);
      }
    }
    if (lane == 0) wout[0][wv] = taken, wout[1][wv] = placed, wout[2][wv] = refused;
  }
  __syncthreads();
  taken = 0;
#pragma unroll
  for (int w = 0; w < ASG_THREADS / 64; ++w) taken = max(taken, wout[0][w]);
  const uint32_t tokens = tot[0], gone = tot[2];
  if (blockIdx.x == 0 && tid == 0) {
    uint32_t placed = 0, refused = 0;
    for (int w = 0; w < ASG_THREADS / 64; ++w) placed = sat_add(placed, wout[1][w]), refused += wout[2][w];
    A.cu_len[R] = (int32_t)tokens;
    A.cursor_out[0] = head + taken;
    A.cursor_out[1] = tail + gone;
    A.counts[0] = (int32_t)placed;
    A.counts[1] = (int32_t)taken;
    A.counts[2] = (int32_t)refused;
    A.counts[3] = (int32_t)gone;
  }

  const uint32_t ps = (uint32_t)A.page_size;
  const uint32_t first = blockIdx.x * ASG_THREADS + tid, step = gridDim.x * ASG_THREADS;
  for (uint32_t t = first; t < (uint32_t)A.max_tokens; t += step) {
    int64_t slot = -1;
    int32_t req = -1, pos = 0, len = 0;
    if (t < tokens) {
      const int i = asg_find(ctok, t);
      uint32_t tok = ctok[i], page = cpage[i];
      int r = i * per;
      AsgReq q = request(r);
      while (t - tok >= q.rows) {  // (the border of thread i + 1 is past t)
        tok = sat_add(tok, q.rows);
        page = sat_add(page, q.want);
        q = request(++r);
      }
      if (q.fits && (!FLAGS || t - tok < q.add) && (q.want == 0 || sat_add(page, q.want) <= avail) && has_rows(q, tok)) {
        const uint32_t p = q.old + (t - tok), at = asg_page(G, p);
        int32_t id;
        if (at < q.held) {
          id = A.table[(int64_t)r * A.table_stride + at];
        } else {
          const uint32_t c = h0 + page + (at - q.held);
          id = A.ring[c < cap ? c : c - cap];
        }
        slot = id < 0 ? -1 : (int64_t)id * ps + (p - at * ps);
        req = r;
        pos = (int32_t)p;
        len = pos + 1;
      }
    }
    A.slot[t] = slot;
    A.req[t] = req;
    A.pos[t] = pos;
    A.len[t] = len;
  }
  for (uint32_t k = first; k < taken; k += step) {
    const int i = asg_find(cpage, k);
    uint32_t page = cpage[i];
    int r = i * per;
    AsgReq q = request(r);
    while (k - page >= q.want) {
      page = sat_add(page, q.want);
      q = request(++r);
    }
    const uint32_t c = h0 + k;
    A.table[(int64_t)r * A.table_stride + q.held + (k - page)] = A.ring[c < cap ? c : c - cap];
  }
  // (no more than the ring holds: with more the caller's tables share pages)
  for (uint32_t k = first; k < min(gone, cap); k += step) {
    const int i = asg_find(cgone, k);
    uint32_t page = cgone[i];
    int r = i * per;
    AsgReq q = request(r);
    while (k - page >= q.gone) {
      page = sat_add(page, q.gone);
      q = request(++r);
    }
    const uint32_t c = t0 + k;
    A.ring[c < cap ? c : c - cap] = A.table[(int64_t)r * A.table_stride + (k - page)];
  }
}

// ---------------------------------------------------------------------------
// rotary positions and the cache store
// ---------------------------------------------------------------------------

struct RotArgs {
  const double* freq;
  const int32_t* axis;
  const void *q, *k, *v;
  const int32_t* pos;
  const int64_t* slot;
  void *q_out, *kc, *vc;
  int64_t q_stride, k_stride, v_stride, pos_stride, q_out_stride;
  int64_t page_stride, token_stride, head_stride, n_slots;
  int32_t head_dim, n_pairs, n_axes, interleaved, n_heads, n_kv_heads, page_size;
};

// ONCE: read once in the launch (a non-temporal load)
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ void ld_vec(const void* p, int64_t i, float (&o)[V]) {
  if constexpr (V == 4 && sizeof(T) == 4) {
    const GLOBAL f32x4* a = (const GLOBAL f32x4*)((const float*)p + i);
    f32x4 v;
    if constexpr (ONCE)
      v = __builtin_nontemporal_load(a);
    else
      v = *a;
    o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
  } else if constexpr (V == 4) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 v = *(const GLOBAL u32x2*)((const uint16_t*)p + i);
    o[0] = __uint_as_float(v.x << 16), o[1] = __uint_as_float(v.x & 0xFFFF0000u);
    o[2] = __uint_as_float(v.y << 16), o[3] = __uint_as_float(v.y & 0xFFFF0000u);
  } else if constexpr (sizeof(T) == 4) {
    o[0] = ldg((const float*)p + i);
  } else {
    o[0] = bf2f(ldg((const uint16_t*)p + i));
  }
}

template <typename T, int V>
__device__ __forceinline__ void st_vec(void* p, int64_t i, const float (&o)[V]) {
  if constexpr (V == 4 && sizeof(T) == 4) {
    stg4((float*)p + i, f32x4{o[0], o[1], o[2], o[3]});
  } else if constexpr (V == 4) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    *(GLOBAL u32x2*)((uint16_t*)p + i) =
        u32x2{pack_bf2(__float_as_uint(o[0]), __float_as_uint(o[1])),
              pack_bf2(__float_as_uint(o[2]), __float_as_uint(o[3]))};
  } else if constexpr (sizeof(T) == 4) {
    *((GLOBAL float*)p + i) = o[0];
  } else {
    *((GLOBAL uint16_t*)p + i) = (uint16_t)pack_bf2(__float_as_uint(o[0]), 0);
  }
}

// One work-group per token and part of its units. The angles' turns
// (pos freq / 2 pi) are reduced in fp64 once per token into LDS and used by
// every head, so what is left is one read and one write of q, k and v: bound by
// HBM for many tokens (8191 tokens, fp32 to bf16: 62.6 us, 4.8 TB/s, the rate of
// a large copy; with plain loads 65.8), by latency for few (1 token 2.5 us, 128
// tokens 3.5). A unit is V elements copied, V pairs of a head split in halves,
// or V / 2 adjacent pairs. One element an access, where halves or rows do not
// start on four: 8191 tokens, 100 of 128 elements in halves 109 us, 96 of them 65.
template <typename S, typename D, int V>
__global__ __launch_bounds__(256) void k_rotary_store(RotArgs A) {
  __shared__ float cs[128], sn[128];
  const int64_t t = blockIdx.x;
  const int n = A.n_pairs;
  if ((int)threadIdx.x < n) {
    const int ax = A.axis ? A.axis[threadIdx.x] : 0;
    const int p = A.pos[(ax > 0 && ax < A.n_axes ? ax : 0) * A.pos_stride + t];
    const double turns = (double)p * (A.freq[threadIdx.x] * 0.15915494309189533577);
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    cs[threadIdx.x] = c;
    sn[threadIdx.x] = s;
  }
  const int64_t slot = A.slot[t];
  const bool store = slot >= 0 && slot < A.n_slots;
  int64_t crow = 0;
  if (store) {
    const int64_t page = slot / A.page_size;
    crow = page * A.page_stride + (slot - page * A.page_size) * A.token_stride;
  }
  __syncthreads();
  const int hd = A.head_dim, rd = 2 * n;
  const int ur = (A.interleaved ? (V == 1 ? n : rd / V) : n / V), per = ur + (hd - rd) / V, pv = hd / V;
  const int nq = A.n_heads * per, nk = nq + A.n_kv_heads * per, all = nk + A.n_kv_heads * pv;
  for (int u = blockIdx.y * 256 + threadIdx.x; u < all; u += gridDim.y * 256) {
    const void* src;
    void* dst;
    int64_t si, di;
    int at;  // unit inside the head; past `ur`: copied elements
    bool put = true;
    if (u < nq) {
      const int h = u / per;
      at = u - h * per;
      src = A.q, si = t * A.q_stride + (int64_t)h * hd;
      dst = A.q_out, di = t * A.q_out_stride + (int64_t)h * hd;
    } else if (u < nk) {
      const int h = (u - nq) / per;
      at = u - nq - h * per;
      src = A.k, si = t * A.k_stride + (int64_t)h * hd;
      dst = A.kc, di = crow + h * A.head_stride, put = store;
    } else {
      const int h = (u - nk) / pv;
      at = u - nk - h * pv + ur - rd / V;  // (element 0 of a copied head)
      src = A.v, si = t * A.v_stride + (int64_t)h * hd;
      dst = A.vc, di = crow + h * A.head_stride, put = store;
    }
    if (!put) continue;
    float a[V], b[V];
    if (u >= nk || at >= ur) {
      const int e = rd + (at - ur) * V;
      ld_vec<S, V, true>(src, si + e, a);
      st_vec<D, V>(dst, di + e, a);
    } else if (A.interleaved) {
      if constexpr (V == 4) {
        ld_vec<S, V, true>(src, si + 4 * at, a);
        const float c0 = cs[2 * at], s0 = sn[2 * at], c1 = cs[2 * at + 1], s1 = sn[2 * at + 1];
        b[0] = a[0] * c0 - a[1] * s0, b[1] = a[0] * s0 + a[1] * c0;
        b[2] = a[2] * c1 - a[3] * s1, b[3] = a[2] * s1 + a[3] * c1;
        st_vec<D, V>(dst, di + 4 * at, b);
      } else {
        float x[1], y[1];
        ld_vec<S, 1>(src, si + 2 * at, x);
        ld_vec<S, 1>(src, si + 2 * at + 1, y);
        const float o0[1] = {x[0] * cs[at] - y[0] * sn[at]}, o1[1] = {x[0] * sn[at] + y[0] * cs[at]};
        st_vec<D, 1>(dst, di + 2 * at, o0);
        st_vec<D, 1>(dst, di + 2 * at + 1, o1);
      }
    } else {
      ld_vec<S, V, true>(src, si + V * at, a);
      ld_vec<S, V, true>(src, si + n + V * at, b);
      float x[V], y[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float c = cs[V * at + i], s = sn[V * at + i];
        x[i] = a[i] * c - b[i] * s;
        y[i] = a[i] * s + b[i] * c;
      }
      st_vec<D, V>(dst, di + V * at, x);
      st_vec<D, V>(dst, di + n + V * at, y);
    }
  }
}

// ---------------------------------------------------------------------------
// the norms around the residual
// ---------------------------------------------------------------------------

struct NormArgs {
  const void *y, *h;
  const float* gate;
  void *h_out, *x;
  const float *post_w, *post_b, *pre_w, *pre_b;
  int64_t y_stride, h_stride, gate_stride, h_out_stride, x_stride;
  int32_t y_bf, h_bf, x_bf, kind, post, d;
  float eps, h_scale, y_scale, inv_d;
};

// Sum over the work-group's up to 16 waves; `red` is a buffer of its own for
// each call. Row shifts and broadcasts inside the wave, then the waves' sums
// in every 16 lanes.
__device__ __forceinline__ float group_sum(float v, float* red) {
#define STEP(ctrl, rows) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, rows, 0xF, false))
  STEP(0x111, 0xF);
  STEP(0x112, 0xF);
  STEP(0x114, 0xF);
  STEP(0x118, 0xF);
  STEP(0x142, 0xA);
  STEP(0x143, 0xC);
  if ((threadIdx.x & 63) == 63) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = (threadIdx.x & 15) < (blockDim.x >> 6) ? red[threadIdx.x & 15] : 0.f;
  STEP(0x111, 0xF);
  STEP(0x112, 0xF);
  STEP(0x114, 0xF);
  STEP(0x118, 0xF);
#undef STEP
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 15));
}

template <int V>
__device__ __forceinline__ void ld_any(const void* p, int bf, int64_t i, float (&o)[V]) {
  if (bf)
    ld_vec<uint16_t, V>(p, i, o);
  else
    ld_vec<float, V>(p, i, o);
}
template <int V>
__device__ __forceinline__ void st_any(void* p, int bf, int64_t i, const float (&o)[V]) {
  if (bf)
    st_vec<uint16_t, V>(p, i, o);
  else
    st_vec<float, V>(p, i, o);
}

// A vector's units of this thread, `fill` where it is null. EARLY: asked for
// with the row, not after its sums.
template <bool EARLY, int V, int N>
struct NormVec {
  const float* p;
  float fill;
  float r[EARLY ? N : 1][V];

  __device__ __forceinline__ NormVec(const float* q, float f, bool used, int units) : p(q), fill(f) {
    if constexpr (EARLY) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int i = 0; i < V; ++i) r[k][i] = fill;
        const int u = threadIdx.x + k * blockDim.x;
        if (p && used && u < units) ld_vec<float, V>(p, (int64_t)u * V, r[k]);
      }
    }
  }
  __device__ __forceinline__ void get(int k, int u, float (&o)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = EARLY ? r[EARLY ? k : 0][i] : fill;
    if constexpr (!EARLY)
      if (p) ld_vec<float, V>(p, (int64_t)u * V, o);
  }
};

template <bool EARLY, int V, int N>
__device__ __forceinline__ void norm_row(float (&v)[N][V], const NormArgs& A, const NormVec<EARLY, V, N>& w,
                                         const NormVec<EARLY, V, N>& b, float (*red)[16]) {
  const int tid = threadIdx.x, th = blockDim.x, units = A.d / V;
  if (A.kind == SCUTE_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) s += v[k][i];
    const float mu = group_sum(s, red[0]) * A.inv_d;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = tid + k * th < units ? v[k][i] - mu : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) s += v[k][i] * v[k][i];
  const float r = rsqrtf(group_sum(s, red[1]) * A.inv_d + A.eps);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int u = tid + k * th;
    if (u < units) {
      float g[V], c[V];
      w.get(k, u, g);
      b.get(k, u, c);
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = v[k][i] * r * g[i] + c[i];
    }
  }
}

// One work-group per row, the row in registers (N units of V elements a
// thread, zeros past its end): y and h are read once, h' and x written once.
// Short rows' vectors are asked for with the row. Bound by HBM for many rows
// (8191 rows of 4096 with a gate for each: 114 us, 5.3 TB/s), by latency for few
// (128 rows: 4.0 us). One element an access, where a row's length or start does
// not allow four: 8191 rows of 4095 163 us, of 4096 72.
template <int V, int N>
__global__ __launch_bounds__(1024) void k_residual_norm(NormArgs A) {
  constexpr bool EARLY = V * N <= 8;
  __shared__ float red[4][16];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, th = blockDim.x, units = A.d / V;
  float v[N][V], h[N][V];
  const bool post = A.y && A.post;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int u = tid + k * th;
#pragma unroll
    for (int i = 0; i < V; ++i) v[k][i] = h[k][i] = 0.f;
    if (u < units) {
      if (A.y) ld_any<V>(A.y, A.y_bf, row * A.y_stride + (int64_t)u * V, v[k]);
      ld_any<V>(A.h, A.h_bf, row * A.h_stride + (int64_t)u * V, h[k]);
    }
  }
  using Vec = NormVec<EARLY, V, N>;
  const Vec pw(A.post_w, 1.f, post, units), pb(A.post_b, 0.f, post, units);
  const Vec gate(A.gate ? A.gate + row * A.gate_stride : nullptr, 1.f, true, units);
  const Vec ew(A.pre_w, 1.f, A.x != nullptr, units), eb(A.pre_b, 0.f, A.x != nullptr, units);
  if (post) norm_row<EARLY, V, N>(v, A, pw, pb, red);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int u = tid + k * th;
    if (u < units) {
      float g[V];
      gate.get(k, u, g);
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = A.h_scale * h[k][i] + (A.y ? A.y_scale * (v[k][i] * g[i]) : 0.f);
      if (A.h_out) st_any<V>(A.h_out, A.h_bf, row * A.h_out_stride + (int64_t)u * V, v[k]);
    }
  }
  if (!A.x) return;
  norm_row<EARLY, V, N>(v, A, ew, eb, red + 2);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int u = tid + k * th;
    if (u < units) st_any<V>(A.x, A.x_bf, row * A.x_stride + (int64_t)u * V, v[k]);
  }
}

// Rows too long for registers an element at a time (over 8192 of a length or
// alignment that does not allow four): every pass computes the elements anew
// from y and h, which stay in the L2 (2000 rows of 9001: 221 us; of 9000, in
// registers: 55).
__global__ __launch_bounds__(1024) void k_residual_norm_long(NormArgs A) {
  __shared__ float red[4][16];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, th = blockDim.x;
  const bool post = A.y && A.post, layer = A.kind == SCUTE_NORM_LAYER;
  const auto at = [](const void* p, int bf, int64_t i) {
    float o[1];
    ld_any<1>(p, bf, i, o);
    return o[0];
  };
  const auto y = [&](int u) { return at(A.y, A.y_bf, row * A.y_stride + u); };
  float mu = 0.f, r = 1.f, s = 0.f;
  if (post) {
    if (layer) {
      for (int u = tid; u < A.d; u += th) s += y(u);
      mu = group_sum(s, red[0]) * A.inv_d;
    }
    s = 0.f;
    for (int u = tid; u < A.d; u += th) s += (y(u) - mu) * (y(u) - mu);
    r = rsqrtf(group_sum(s, red[1]) * A.inv_d + A.eps);
  }
  const auto h1 = [&](int u) {  // h'
    float z = 0.f;
    if (A.y) {
      z = (y(u) - mu) * r;
      if (post) z = z * (A.post_w ? ldg(A.post_w + u) : 1.f) + (A.post_b ? ldg(A.post_b + u) : 0.f);
      z *= A.y_scale * (A.gate ? ldg(A.gate + row * A.gate_stride + u) : 1.f);
    }
    return A.h_scale * at(A.h, A.h_bf, row * A.h_stride + u) + z;
  };
  float m1 = 0.f, r1 = 1.f;
  if (A.x) {
    if (layer) {
      s = 0.f;
      for (int u = tid; u < A.d; u += th) s += h1(u);
      m1 = group_sum(s, red[2]) * A.inv_d;
    }
    s = 0.f;
    for (int u = tid; u < A.d; u += th) s += (h1(u) - m1) * (h1(u) - m1);
    r1 = rsqrtf(group_sum(s, red[3]) * A.inv_d + A.eps);
  }
  for (int u = tid; u < A.d; u += th) {  // (h_out may be h: an element is read before it is written)
    const float v[1] = {h1(u)};
    if (A.h_out) st_any<1>(A.h_out, A.h_bf, row * A.h_out_stride + u, v);
    if (A.x) {
      const float o[1] = {(v[0] - m1) * r1 * (A.pre_w ? ldg(A.pre_w + u) : 1.f) + (A.pre_b ? ldg(A.pre_b + u) : 0.f)};
      st_any<1>(A.x, A.x_bf, row * A.x_stride + u, o);
    }
  }
}

}  // namespace scute

using namespace scute;

// ---------------------------------------------------------------------------
// entry points
// ---------------------------------------------------------------------------

namespace {

bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

// work-groups of `threads` that one launch may have in x (2^32 - 1 threads)
int64_t most_groups(int threads) { return 0xFFFFFFFFll / threads; }

scute_status launched(const char* fn) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SCUTE_OK : hip_fail(e, fn);
}

}  // namespace

extern "C" scute_status scute_cache_assign(const scute_cache_assign_args* A, void* stream) {
  const char* fn = "scute_cache_assign";
  if (!A) return fail(SCUTE_E_INVALID, "scute_cache_assign: args is null");
  if (A->device < 0) return fail(SCUTE_E_INVALID, "scute_cache_assign: device must be >= 0");
  if (A->n_requests < 0 || A->n_requests > 65536)
    return fail(SCUTE_E_SHAPE, "scute_cache_assign: n_requests must be in [0, 65536]");
  if (A->page_size < 1 || A->page_size > 65536)
    return fail(SCUTE_E_SHAPE, "scute_cache_assign: page_size must be in [1, 65536]");
  if (A->table_width < 1 || A->table_width > (1 << 24) || A->table_stride < A->table_width ||
      A->table_stride > ((int64_t)1 << 40))
    return fail(SCUTE_E_SHAPE, "scute_cache_assign: table_width must be in [1, 2^24] and at most table_stride");
  if (A->ring_size < 1 || A->ring_size > (1 << 30))
    return fail(SCUTE_E_SHAPE, "scute_cache_assign: ring_size must be in [1, 2^30]");
  if (A->max_tokens < 0 || A->max_tokens > (1 << 30))
    return fail(SCUTE_E_SHAPE, "scute_cache_assign: max_tokens must be in [0, 2^30]");
  const bool some = A->n_requests > 0;
  if (!A->ring || !A->cursor || !A->cursor_out || !A->cu_len || !A->counts ||
      (some && (!A->old_len || !A->new_len || !A->table || !A->seq_len)) ||
      (A->max_tokens > 0 && (!A->slot || !A->req || !A->pos || !A->len)))
    return fail(SCUTE_E_INVALID, "scute_cache_assign: null pointer");
  for (const void* p : {(const void*)A->old_len, (const void*)A->new_len, (const void*)A->table,
                        (const void*)A->ring, (const void*)A->seq_len, (const void*)A->cu_len,
                        (const void*)A->req, (const void*)A->pos, (const void*)A->len, (const void*)A->counts})
    if (misaligned(p, 4)) return fail(SCUTE_E_INVALID, "scute_cache_assign: misaligned pointer");
  for (const void* p : {(const void*)A->cursor, (const void*)A->cursor_out, (const void*)A->slot})
    if (misaligned(p, 8)) return fail(SCUTE_E_INVALID, "scute_cache_assign: misaligned pointer");
  if (A->flags & ~(uint32_t)(SCUTE_ASSIGN_FIT_ROWS | SCUTE_ASSIGN_ONE_EACH))
    return fail(SCUTE_E_INVALID, "scute_cache_assign: unknown flag");
  if ((A->flags & SCUTE_ASSIGN_ONE_EACH) && A->max_tokens < A->n_requests)
    return fail(SCUTE_E_SHAPE, "scute_cache_assign: a row for each request needs max_tokens >= n_requests");
  // work-groups read the inputs while others write the outputs
  struct Range {
    const void* p;
    int64_t bytes;
  };
  const int64_t R = A->n_requests, T = A->max_tokens;
  const Range ins[] = {{A->cursor, 16}, {some ? A->old_len : nullptr, 4 * R}, {some ? A->new_len : nullptr, 4 * R}};
  const Range outs[] = {{A->cursor_out, 16}, {some ? A->seq_len : nullptr, 4 * R}, {A->cu_len, 4 * (R + 1)}, {A->counts, 16},
                        {T ? A->slot : nullptr, 8 * T}, {T ? A->req : nullptr, 4 * T}, {T ? A->pos : nullptr, 4 * T},
                        {T ? A->len : nullptr, 4 * T}, {A->ring, 4 * (int64_t)A->ring_size}};
  for (const Range& o : outs) {
    for (const Range& i : ins)
      if (rows_meet(o.p, 0, o.bytes, i.p, 0, i.bytes, 1))
        return fail(SCUTE_E_INVALID, "scute_cache_assign: an output is also an input");
    for (const Range* b = outs; b < &o; ++b)
      if (rows_meet(o.p, 0, o.bytes, b->p, 0, b->bytes, 1))
        return fail(SCUTE_E_INVALID, "scute_cache_assign: outputs overlap");
  }
  OnDevice g(A->device);
  if (!g.ok()) return hip_fail(g.err, fn);
  AsgArgs G{*A, 0, 0};
  while ((1 << G.shift) < A->page_size) ++G.shift;
  G.mul = (uint32_t)((((uint64_t)1 << (31 + G.shift)) + A->page_size - 1) / A->page_size);
  // one round of the tokens over up to 512 work-groups; at least one work-group
  // for every 256 requests, whose pages may have to be copied
  const int64_t work = std::max<int64_t>(A->max_tokens, 4 * (int64_t)A->n_requests);
  const int64_t blocks = std::min<int64_t>(std::max<int64_t>(1, (work + ASG_THREADS - 1) / ASG_THREADS), 512);
  if (A->flags)
    hipLaunchKernelGGL(k_cache_assign<true>, dim3((unsigned)blocks), dim3(ASG_THREADS), 0, (hipStream_t)stream, G);
  else
    hipLaunchKernelGGL(k_cache_assign<false>, dim3((unsigned)blocks), dim3(ASG_THREADS), 0, (hipStream_t)stream, G);
  return launched(fn);
}

namespace scute {

scute_status check_cache(const scute_kv_cache* C, const char* fn) {
  const std::string f(fn);
  if (!C) return fail(SCUTE_E_INVALID, f + ": cache is null");
  if (C->device < 0) return fail(SCUTE_E_INVALID, f + ": the cache's device must be >= 0");
  if (C->dtype != SCUTE_BF16 && C->dtype != SCUTE_F32)
    return fail(SCUTE_E_INVALID, f + ": the cache's dtype must be SCUTE_BF16 or SCUTE_F32");
  if (C->page_size < 1 || C->page_size > 65536 || C->n_kv_heads < 1 || C->n_kv_heads > 1024)
    return fail(SCUTE_E_SHAPE, f + ": page_size must be in [1, 65536] and n_kv_heads in [1, 1024]");
  if (C->head_dim < 8 || C->head_dim > 256 || C->head_dim % 8)
    return fail(SCUTE_E_SHAPE, f + ": head_dim must be a multiple of 8 in [8, 256]");
  if (C->n_pages < 1 || C->n_pages > 0x7FFFFFFF)
    return fail(SCUTE_E_SHAPE, f + ": n_pages must be in [1, 2^31 - 1]");
  for (int64_t s : {C->page_stride, C->token_stride, C->head_stride})
    if (s < 8 || s % 8 || s > ((int64_t)1 << 40))
      return fail(SCUTE_E_SHAPE, f + ": the cache's strides must be multiples of 8 in [8, 2^40]");
  if (C->token_stride >= (1 << 24)) return fail(SCUTE_E_SHAPE, f + ": token_stride must be below 2^24");
  if (!C->k || !C->v || misaligned(C->k, 16) || misaligned(C->v, 16))
    return fail(SCUTE_E_INVALID, f + ": the cache's k and v must be 16-byte aligned pointers");
  return SCUTE_OK;
}

}  // namespace scute

extern "C" scute_status scute_rotary_store(const scute_rotary* Ro, const scute_kv_cache* C, const void* q,
                                           int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                           int64_t v_stride, int32_t src_dtype, const int32_t* pos,
                                           int64_t pos_stride, const int64_t* slot, int32_t n_tokens,
                                           int32_t n_heads, void* q_out, int64_t q_out_stride, void* stream) {
  const char* fn = "scute_rotary_store";
  if (!Ro) return fail(SCUTE_E_INVALID, "scute_rotary_store: rotary is null");
  scute_status st = check_cache(C, fn);
  if (st != SCUTE_OK) return st;
  if (Ro->head_dim != C->head_dim)
    return fail(SCUTE_E_SHAPE, "scute_rotary_store: the rotary's and the cache's head_dim differ");
  if (Ro->rot_dim < 0 || Ro->rot_dim > Ro->head_dim || Ro->rot_dim % 2)
    return fail(SCUTE_E_SHAPE, "scute_rotary_store: rot_dim must be even and in [0, head_dim]");
  if (Ro->n_axes < 1 || Ro->n_axes > 8) return fail(SCUTE_E_SHAPE, "scute_rotary_store: n_axes must be in [1, 8]");
  if (Ro->interleaved != 0 && Ro->interleaved != 1)
    return fail(SCUTE_E_INVALID, "scute_rotary_store: interleaved must be 0 or 1");
  if (src_dtype != SCUTE_F32 && src_dtype != SCUTE_BF16)
    return fail(SCUTE_E_INVALID, "scute_rotary_store: src_dtype must be SCUTE_F32 or SCUTE_BF16");
  if (n_tokens < 0 || n_heads < 1 || n_heads > 65536)
    return fail(SCUTE_E_SHAPE, "scute_rotary_store: n_tokens must be >= 0 and n_heads in [1, 65536]");
  const int64_t hd = C->head_dim, big = (int64_t)1 << 40;
  for (int64_t s : {q_stride, k_stride, v_stride, q_out_stride, pos_stride})
    if (s < 0 || s > big) return fail(SCUTE_E_SHAPE, "scute_rotary_store: strides must be in [0, 2^40]");
  if (n_tokens > 1 && q_out_stride < n_heads * hd)
    return fail(SCUTE_E_SHAPE, "scute_rotary_store: rows of q_out overlap");
  if (n_tokens == 0) return SCUTE_OK;
  if (!q || !k || !v || !slot || !q_out || (Ro->rot_dim && (!pos || !Ro->freq)))
    return fail(SCUTE_E_INVALID, "scute_rotary_store: null pointer");
  const uintptr_t es = src_dtype == SCUTE_F32 ? 4 : 2, ed = C->dtype == SCUTE_F32 ? 4 : 2;
  if (misaligned(q, es) || misaligned(k, es) || misaligned(v, es) || misaligned(q_out, ed) || misaligned(pos, 4) ||
      misaligned(slot, 8) || misaligned(Ro->freq, 8) || misaligned(Ro->axis, 4))
    return fail(SCUTE_E_INVALID, "scute_rotary_store: misaligned pointer");
  const int64_t wq = n_heads * hd, wk = C->n_kv_heads * hd, si = (int64_t)es, so = (int64_t)ed, T = n_tokens;
  const bool same = q == q_out && es == ed && (T == 1 || q_stride == q_out_stride);
  if ((!same && rows_meet(q, q_stride * si, wq * si, q_out, q_out_stride * so, wq * so, T)) ||
      rows_meet(k, k_stride * si, wk * si, q_out, q_out_stride * so, wq * so, T) ||
      rows_meet(v, v_stride * si, wk * si, q_out, q_out_stride * so, wq * so, T) || (q == q_out && !same))
    return fail(SCUTE_E_INVALID, "scute_rotary_store: q_out overlaps q (of another type or stride), k or v");
  OnDevice g(C->device);
  if (!g.ok()) return hip_fail(g.err, fn);

  const int n = Ro->rot_dim / 2;
  RotArgs A{Ro->freq, Ro->axis, q, k, v, pos, slot, q_out, C->k, C->v, q_stride, k_stride, v_stride, pos_stride,
                  q_out_stride, C->page_stride, C->token_stride, C->head_stride, C->n_pages * C->page_size,
                  C->head_dim, n, Ro->n_axes, Ro->interleaved, n_heads, C->n_kv_heads, C->page_size};
  // four elements an access where every row's accesses are aligned to them and
  // no unit crosses the rotated part's halves or end
  const bool vec = ((q_stride | k_stride | v_stride | q_out_stride) % 4 == 0) && !misaligned(q, 4 * es) &&
                   !misaligned(k, 4 * es) && !misaligned(v, 4 * es) && !misaligned(q_out, 4 * ed) &&
                   (Ro->interleaved ? n % 2 == 0 : n % 4 == 0);
  const int V = vec ? 4 : 1;
  const int64_t rot = Ro->interleaved && V == 4 ? 2 * n / V : n / V;
  const int64_t units = (n_heads + C->n_kv_heads) * (rot + (hd - 2 * n) / V) + C->n_kv_heads * (hd / V);
  // few tokens: their units spread over more work-groups, one unit a thread
  const int64_t parts = std::min<int64_t>(std::min<int64_t>((units + 255) / 256, 4096),
                                          std::max<int64_t>(1, 1024 / n_tokens));
  const hipStream_t s = (hipStream_t)stream;
  for (int64_t t = 0; t < n_tokens; t += most_groups(256)) {
    const dim3 grid((unsigned)std::min(most_groups(256), n_tokens - t), (unsigned)parts);
    A.q = (const char*)q + t * q_stride * (int64_t)es;
    A.k = (const char*)k + t * k_stride * (int64_t)es;
    A.v = (const char*)v + t * v_stride * (int64_t)es;
    A.q_out = (char*)q_out + t * q_out_stride * (int64_t)ed;
    A.pos = pos ? pos + t : nullptr;
    A.slot = slot + t;
#define ROT(S, D)                                                                    \
  do {                                                                               \
    if (vec)                                                                         \
      hipLaunchKernelGGL((k_rotary_store<S, D, 4>), grid, dim3(256), 0, s, A);       \
    else                                                                             \
      hipLaunchKernelGGL((k_rotary_store<S, D, 1>), grid, dim3(256), 0, s, A);       \
  } while (0)
    if (es == 4 && ed == 4)
      ROT(float, float);
    else if (es == 4)
      ROT(float, uint16_t);
    else if (ed == 4)
      ROT(uint16_t, float);
    else
      ROT(uint16_t, uint16_t);
#undef ROT
    const scute_status ls = launched(fn);
    if (ls != SCUTE_OK) return ls;
  }
  return SCUTE_OK;
}

extern "C" scute_status scute_residual_norm(const scute_norm* N, const void* y, int32_t y_dtype, int64_t y_stride,
                                            const void* h, int32_t h_dtype, int64_t h_stride, const float* gate,
                                            int64_t gate_stride, void* h_out, int64_t h_out_stride, void* x,
                                            int32_t x_dtype, int64_t x_stride, int32_t n_rows, void* stream) {
  const char* fn = "scute_residual_norm";
  if (!N) return fail(SCUTE_E_INVALID, "scute_residual_norm: norm is null");
  if (N->device < 0) return fail(SCUTE_E_INVALID, "scute_residual_norm: device must be >= 0");
  if (N->kind != SCUTE_NORM_RMS && N->kind != SCUTE_NORM_LAYER)
    return fail(SCUTE_E_INVALID, "scute_residual_norm: kind must be SCUTE_NORM_RMS or SCUTE_NORM_LAYER");
  if (N->d < 1 || N->d > 32768) return fail(SCUTE_E_SHAPE, "scute_residual_norm: d must be in [1, 32768]");
  if (n_rows < 0) return fail(SCUTE_E_SHAPE, "scute_residual_norm: n_rows must be >= 0");
  auto bad = [](int32_t dt) { return dt != SCUTE_F32 && dt != SCUTE_BF16; };
  if (bad(h_dtype) || (y && bad(y_dtype)) || (x && bad(x_dtype)))
    return fail(SCUTE_E_INVALID, "scute_residual_norm: types must be SCUTE_F32 or SCUTE_BF16");
  const int64_t big = (int64_t)1 << 40;
  for (int64_t s : {y_stride, h_stride, gate_stride, h_out_stride, x_stride})
    if (s < 0 || s > big) return fail(SCUTE_E_SHAPE, "scute_residual_norm: strides must be in [0, 2^40]");
  if (n_rows > 1 && ((h_out && h_out_stride < N->d) || (x && x_stride < N->d)))
    return fail(SCUTE_E_SHAPE, "scute_residual_norm: rows of an output overlap");
  if (n_rows == 0) return SCUTE_OK;
  if (!h_out && !x) return fail(SCUTE_E_INVALID, "scute_residual_norm: h_out and x are null");
  if (!h) return fail(SCUTE_E_INVALID, "scute_residual_norm: h is null");
  const uintptr_t ey = y_dtype == SCUTE_F32 ? 4 : 2, eh = h_dtype == SCUTE_F32 ? 4 : 2, ex = x_dtype == SCUTE_F32 ? 4 : 2;
  if (misaligned(y, ey) || misaligned(h, eh) || misaligned(h_out, eh) || misaligned(x, ex))
    return fail(SCUTE_E_INVALID, "scute_residual_norm: misaligned pointer");
  struct Rows {
    const void* p;
    int64_t stride, es;
  };
  const Rows ry{y, y_stride, (int64_t)ey}, rh{h, h_stride, (int64_t)eh}, rg{gate, gate_stride, 4};
  const Rows rho{h_out, h_out_stride, (int64_t)eh}, rx{x, x_stride, (int64_t)ex};
  const auto meet = [&](const Rows& a, const Rows& b) {
    return a.p && (a.p == b.p || rows_meet(a.p, a.stride * a.es, N->d * a.es, b.p, b.stride * b.es, N->d * b.es, n_rows));
  };
  if (meet(rx, rh) || meet(rx, ry) || meet(rx, rho) || meet(rx, rg))
    return fail(SCUTE_E_INVALID, "scute_residual_norm: x is also h, y, gate or h_out");
  const bool in_place = h_out == h && (n_rows == 1 || h_out_stride == h_stride);
  if (meet(rho, ry) || meet(rho, rg) || (!in_place && meet(rho, rh)))
    return fail(SCUTE_E_INVALID, "scute_residual_norm: h_out is also y or gate, or h at another place or stride");
  bool vec = N->d % 4 == 0 && ((y_stride | h_stride | gate_stride | h_out_stride | x_stride) % 4 == 0) &&
             !misaligned(y, 4 * ey) && !misaligned(h, 4 * eh) && !misaligned(h_out, 4 * eh) && !misaligned(x, 4 * ex);
  for (const float* p : {gate, N->post_w, N->post_b, N->pre_w, N->pre_b}) {
    if (misaligned(p, 4)) return fail(SCUTE_E_INVALID, "scute_residual_norm: misaligned pointer");
    vec = vec && !misaligned(p, 16);
  }
  OnDevice g(N->device);
  if (!g.ok()) return hip_fail(g.err, fn);

  NormArgs A{y, h, gate, h_out, x, N->post_w, N->post_b, N->pre_w, N->pre_b, y_stride, h_stride, gate_stride,
                   h_out_stride, x_stride, y_dtype == SCUTE_BF16, h_dtype == SCUTE_BF16, x_dtype == SCUTE_BF16,
                   N->kind, N->post, N->d, N->eps, N->h_scale, N->y_scale, 1.f / (float)N->d};
  const int V = vec ? 4 : 1, units = N->d / V;
  // a unit a thread for few rows (128 rows of 4096: 4.4 us with 1024 threads,
  // 4.9 with 512), more of them for many (8191 rows of 4096: 138 us with 1024,
  // 114 with 512, 122 with 256), where other rows hide a row's latencies
  const int most = n_rows <= 512 || units > 512 * 8 ? 1024 : 512;
  int threads = 64;
  while (threads < most && units > threads) threads *= 2;
  const int per = (units + threads - 1) / threads;  // at most 8 of 4 elements, 32 of one
  const hipStream_t s = (hipStream_t)stream;
  for (int64_t r = 0; r < n_rows; r += most_groups(threads)) {
    const dim3 grid((unsigned)std::min(most_groups(threads), n_rows - r));
    A.y = y ? (const char*)y + r * y_stride * (int64_t)ey : nullptr;
    A.h = (const char*)h + r * h_stride * (int64_t)eh;
    A.gate = gate ? gate + r * gate_stride : nullptr;
    A.h_out = h_out ? (char*)h_out + r * h_out_stride * (int64_t)eh : nullptr;
    A.x = x ? (char*)x + r * x_stride * (int64_t)ex : nullptr;
#define NORM(VV, NN) hipLaunchKernelGGL((k_residual_norm<VV, NN>), grid, dim3(threads), 0, s, A)
    if (vec) {
      if (per <= 1) NORM(4, 1);
      else if (per <= 2) NORM(4, 2);
      else if (per <= 4) NORM(4, 4);
      else NORM(4, 8);
    } else {
      if (per <= 1) NORM(1, 1);
      else if (per <= 4) NORM(1, 4);
      else if (per <= 8) NORM(1, 8);
      else hipLaunchKernelGGL(k_residual_norm_long, grid, dim3(threads), 0, s, A);
    }
#undef NORM
    const scute_status ls = launched(fn);
    if (ls != SCUTE_OK) return ls;
  }
  return SCUTE_OK;
}
