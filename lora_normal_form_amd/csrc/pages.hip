// Requests that share pages: pages of requests that go on from others
// (scute_cache_fork), copies of pages (scute_cache_copy) and positions of a
// request moved together (scute_cache_compact).

#include <algorithm>

#include "block.h"
#include "kernels.h"

namespace scute {

// ---------------------------------------------------------------------------
// pages of requests that go on from others
// ---------------------------------------------------------------------------

// Who holds a page after the step follows from the tables alone, so nothing is
// counted between steps: every entry marks its page (held before; held wholly
// after; the first request that holds it partly), the marks say which last pages
// are to be copied and which pages are free, and two prefix sums number those.
// Three launches: marks, sums of blocks, and the tables and the ring, each a chain
// of four to six reads that wait for one another, which is what bounds them. Marks are
// plain stores of one value, but for the first partial holder, an atomic maximum
// of n_requests - r, so the order of the stores does not matter.
constexpr int FORK_THREADS = 1024, FORK_PAGES = 4 * FORK_THREADS;  // pages a block

struct ForkArgs {
  scute_cache_fork_args a;
  uint32_t mul, shift;  // x / page_size = x mul >> 31 + shift for x < 2^31
  int32_t* first;       // [n_pages] n_requests - r of the first request that holds the page partly (0: none)
  uint8_t *whole, *before;  // [n_pages] held wholly after, held before
  uint32_t* need;       // [n_requests] copies wanted by the requests before it in its block; FORK_WANTS: it wants one
  uint32_t *need_sum, *free_sum;  // of each block
  int32_t req_blocks, page_blocks, row_parts;
};
constexpr uint32_t FORK_WANTS = 1u << 31, FORK_LEN = 1u << 30;

__device__ __forceinline__ uint32_t fork_div(const ForkArgs& G, uint32_t x) {
  return (uint32_t)(((uint64_t)x * G.mul) >> (31 + G.shift));
}
// positions that a request's table row can hold, of its length
__device__ __forceinline__ uint32_t fork_len(const ForkArgs& G, int32_t len) {
  const uint64_t room = (uint64_t)G.a.table_width * G.a.page_size;
  const uint32_t n = len > 0 ? min((uint32_t)len, FORK_LEN) : 0u;
  return room < n ? (uint32_t)room : n;
}
struct ForkReq {
  int parent;
  uint32_t n, whole, part, cols;      // positions, whole pages, positions on the last, columns of the table
  uint32_t drop_from, drop_to;        // columns that are dropped
};
// of the request that goes on from the first n positions of `parent`
__device__ __forceinline__ ForkReq fork_req(const ForkArgs& G, int parent, uint32_t n) {
  const scute_cache_fork_args& A = G.a;
  ForkReq q;
  q.parent = parent, q.n = n;
  q.whole = fork_div(G, q.n);
  q.part = q.n - q.whole * A.page_size;
  q.cols = q.whole + (q.part ? 1u : 0u);
  q.drop_from = q.drop_to = 0;
  if (A.window > 0 && q.n > (uint32_t)A.window) {  // pages whose positions all lie in [sinks, n - window)
    const uint32_t ps = (uint32_t)A.page_size, s = (uint32_t)A.sinks;
    q.drop_from = s > FORK_LEN ? q.cols : fork_div(G, s + ps - 1);
    q.drop_to = fork_div(G, q.n - (uint32_t)A.window);
  }
  return q;
}
__device__ __forceinline__ ForkReq fork_req(const ForkArgs& G, int r) {
  const scute_cache_fork_args& A = G.a;
  int parent = ldg(A.parent + r);
  const bool lives = (uint32_t)parent < (uint32_t)A.n_requests;
  if (!lives) parent = r;
  uint32_t n = lives ? fork_len(G, ldg(A.len + parent)) : 0u;
  if (A.keep) n = min(n, (uint32_t)max(ldg(A.keep + r), 0));
  return fork_req(G, parent, n);
}
// the page of a column of the request after the step, before copies (-1: none)
__device__ __forceinline__ int fork_page(const ForkArgs& G, const ForkReq& q, uint32_t c) {
  if (c >= q.cols || (c >= q.drop_from && c < q.drop_to)) return -1;
  const int p = ldg(G.a.table + (int64_t)q.parent * G.a.table_stride + c);
  return (uint32_t)p < (uint32_t)G.a.n_pages ? p : -1;
}

__global__ __launch_bounds__(256) void k_fork_mark(ForkArgs G) {
  const scute_cache_fork_args& A = G.a;
  for (int r = blockIdx.y; r < A.n_requests; r += gridDim.y) {
    const ForkReq q = fork_req(G, r);
    const uint32_t held = fork_div(G, fork_len(G, ldg(A.len + r)) + A.page_size - 1);
    for (uint32_t c = blockIdx.x * 256 + threadIdx.x; c < max(held, q.cols); c += gridDim.x * 256) {
      if (c < held) {
        const int p = ldg(A.table + (int64_t)r * A.table_stride + c);
        if ((uint32_t)p < (uint32_t)A.n_pages) G.before[p] = 1;
      }
      const int p = fork_page(G, q, c);
      if (p >= 0) {
        if (c < q.whole)
          G.whole[p] = 1;
        else
          atomicMax(G.first + p, A.n_requests - r);
      }
    }
  }
}

// sum over the work-group's 16 waves of v, and what the threads before this one
// add to it
__device__ __forceinline__ uint32_t fork_scan(uint32_t v, uint32_t* s_sum, uint32_t& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint32_t inc = v;
#define STEP(ctrl, rows) inc += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)inc, ctrl, rows, 0xF, false)
  STEP(0x111, 0xF);
  STEP(0x112, 0xF);
  STEP(0x114, 0xF);
  STEP(0x118, 0xF);
  STEP(0x142, 0xA);
  STEP(0x143, 0xC);
#undef STEP
  if (lane == 63) s_sum[w] = inc;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int x = 0; x < FORK_THREADS / 64; ++x) {
    if (x < w) before += s_sum[x];
    total += s_sum[x];
  }
  __syncthreads();  // (s_sum may be used again)
  return before + inc - v;
}

__device__ __forceinline__ bool fork_free(const ForkArgs& G, uint32_t p) {
  return p < (uint32_t)G.a.n_pages && G.before[p] && !G.whole[p] && G.first[p] == 0;
}

__global__ __launch_bounds__(FORK_THREADS) void k_fork_sums(ForkArgs G) {
  const scute_cache_fork_args& A = G.a;
  __shared__ uint32_t s_sum[FORK_THREADS / 64];
  uint32_t total;
  if ((int)blockIdx.x < G.page_blocks) {
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) n += fork_free(G, blockIdx.x * FORK_PAGES + threadIdx.x * 4 + i);
    fork_scan(n, s_sum, total);
    if (threadIdx.x == 0) G.free_sum[blockIdx.x] = total;
  } else {
    const int b = blockIdx.x - G.page_blocks, r = b * FORK_THREADS + threadIdx.x;
    uint32_t wants = 0;
    if (r < A.n_requests) {
      const ForkReq q = fork_req(G, r);
      const int p = q.part ? fork_page(G, q, q.whole) : -1;
      wants = p >= 0 && (G.whole[p] || G.first[p] != A.n_requests - r);
    }
    const uint32_t at = fork_scan(wants, s_sum, total);
    if (r < A.n_requests) G.need[r] = at | (wants ? FORK_WANTS : 0u);
    if (threadIdx.x == 0) G.need_sum[b] = total;
  }
}

__global__ __launch_bounds__(FORK_THREADS) void k_fork_apply(ForkArgs G) {
  const scute_cache_fork_args& A = G.a;
  __shared__ uint32_t s_sum[FORK_THREADS / 64];
  const int tid = threadIdx.x;
  const int64_t head = A.cursor[0], tail = A.cursor[1];
  const uint32_t cap = (uint32_t)A.ring_size;
  const int64_t free64 = tail - head;
  const uint32_t avail = free64 <= 0 ? 0u : free64 < (int64_t)cap ? (uint32_t)free64 : cap;
  const uint32_t h0 = (uint32_t)((uint64_t)head % cap), t0 = (uint32_t)((uint64_t)tail % cap);
  uint32_t total;
  if ((int)blockIdx.x < G.page_blocks) {
    // the block's free pages to the ring, behind those of the blocks before it;
    // the marks are cleared for the next call
    const int b = blockIdx.x;
    uint32_t before = 0;
    for (int i = tid; i < b; i += FORK_THREADS) before += G.free_sum[i];
    fork_scan(before, s_sum, total);
    before = total;
    const uint32_t p0 = b * FORK_PAGES + tid * 4;
    bool gone[4];
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) n += gone[i] = fork_free(G, p0 + i);
    uint32_t at = before + fork_scan(n, s_sum, total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (p0 + i >= (uint32_t)A.n_pages) break;
      if (gone[i]) {
        const uint32_t c = t0 + at;
        if (at < cap) A.ring[c < cap ? c : c - cap] = (int32_t)(p0 + i);  // (no more than the ring holds)
        ++at;
      }
      G.before[p0 + i] = G.whole[p0 + i] = 0;
      G.first[p0 + i] = 0;
    }
    return;
  }
  int b = blockIdx.x - G.page_blocks;
  if (b == 0) {  // cursors and counts
    uint32_t gone = 0, wants = 0, live = 0;
    for (int i = tid; i < G.page_blocks; i += FORK_THREADS) gone += G.free_sum[i];
    for (int i = tid; i < G.req_blocks; i += FORK_THREADS) wants += G.need_sum[i];
    fork_scan(gone, s_sum, total);
    gone = total;
    fork_scan(wants, s_sum, total);
    wants = total;
    uint32_t base = 0;
    for (int i = 0; i < G.req_blocks; ++i) {
      const int r = i * FORK_THREADS + tid;
      if (r < A.n_requests) {
        const ForkReq q = fork_req(G, r);
        const uint32_t at = G.need[r];
        const bool refused = (at & FORK_WANTS) && base + (at & ~FORK_WANTS) >= avail;
        live += (refused ? q.whole : q.n) > 0;
      }
      base += G.need_sum[i];
    }
    fork_scan(live, s_sum, total);
    if (tid == 0) {
      const uint32_t taken = min(wants, avail);
      A.cursor_out[0] = head + taken;
      A.cursor_out[1] = tail + gone;
      A.counts[0] = (int32_t)total;
      A.counts[1] = (int32_t)taken;
      A.counts[2] = (int32_t)(wants - taken);
      A.counts[3] = (int32_t)gone;
    }
    return;
  }
  b -= 1;
  // rows of the table, row_parts work-groups a row
  const int rows = (gridDim.x - G.page_blocks - 1) / G.row_parts, part = b % G.row_parts;
  for (int r = b / G.row_parts; r < A.n_requests; r += rows) {
    const ForkReq q = fork_req(G, r);
    const uint32_t need = G.need[r];
    int last = -2;  // the last page where it is not the parent's: -1 none
    if (need & FORK_WANTS) {  // (uniform)
      uint32_t at = need & ~FORK_WANTS;
      for (int i = 0; i < r / FORK_THREADS; ++i) at += G.need_sum[i];
      const uint32_t c = h0 + at;
      last = at < avail ? ldg(A.ring + (c < cap ? c : c - cap)) : -1;
      if (at < avail && part == 0 && tid == 0) {
        A.src[r] = fork_page(G, q, q.whole);
        A.dst[r] = last;
        A.n[r] = (int32_t)q.part;
      }
      if (at >= avail) last = -3;
    }
    if (part == 0 && tid == 0) {
      A.seq_len[r] = (int32_t)(last == -3 ? q.n - q.part : q.n);
      if (last == -2 || last == -3) A.src[r] = A.dst[r] = -1, A.n[r] = 0;
    }
    for (uint32_t c = part * FORK_THREADS + tid; c < (uint32_t)A.table_width; c += G.row_parts * FORK_THREADS) {
      int p = fork_page(G, q, c);
      if (last != -2 && c == q.whole) p = last == -3 ? -1 : last;
      A.table_out[(int64_t)r * A.table_out_stride + c] = p;
    }
  }
}

// Few requests and pages: one work-group does it in one launch, marks in LDS, a
// thread a request, eight pages a thread, a wave a row. In a graph, with the copies:
// 8 requests of 13 pages 13.3 us (three launches 19.4), 32 of 128 16.8 (22.0), 128
// of 32 20.0 (21.8), 256 of 32, the most pieces, 22.1 (22.3).
constexpr int FORK_ONE_PAGES = 8 * FORK_THREADS, FORK_ONE_PIECES = 256;  // (pieces: of 64 entries of the table)

__global__ __launch_bounds__(FORK_THREADS) void k_fork_one(ForkArgs G) {
  const scute_cache_fork_args& A = G.a;
  __shared__ uint32_t s_before[FORK_ONE_PAGES / 32], s_whole[FORK_ONE_PAGES / 32], s_sum[FORK_THREADS / 64];
  __shared__ int32_t s_first[FORK_ONE_PAGES], s_parent[FORK_ONE_PIECES], s_last[FORK_ONE_PIECES];
  __shared__ uint32_t s_n[FORK_ONE_PIECES], s_held[FORK_ONE_PIECES];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, R = A.n_requests;
  const uint32_t n_pages = (uint32_t)A.n_pages;
  const int64_t head = A.cursor[0], tail = A.cursor[1];
  ForkReq q{};
  if (tid < R) {
    q = fork_req(G, tid);
    s_parent[tid] = q.parent, s_n[tid] = q.n;
    s_held[tid] = fork_div(G, fork_len(G, ldg(A.len + tid)) + A.page_size - 1);
  }
  for (int i = tid; i < FORK_ONE_PAGES; i += FORK_THREADS) s_first[i] = 0;
  if (tid < FORK_ONE_PAGES / 32) s_before[tid] = s_whole[tid] = 0;
  __syncthreads();
  for (int r = w; r < R; r += FORK_THREADS / 64) {
    const ForkReq o = fork_req(G, s_parent[r], s_n[r]);
    const uint32_t held = s_held[r];
    for (uint32_t c = lane; c < max(held, o.cols); c += 64) {
      const int was = c < held ? ldg(A.table + (int64_t)r * A.table_stride + c) : -1, p = fork_page(G, o, c);
      if ((uint32_t)was < n_pages) atomicOr(s_before + was / 32, 1u << (was % 32));
      if (p >= 0) {
        if (c < o.whole)
          atomicOr(s_whole + p / 32, 1u << (p % 32));
        else
          atomicMax(s_first + p, R - r);
      }
    }
  }
  __syncthreads();
  const uint32_t cap = (uint32_t)A.ring_size;
  const int64_t free64 = tail - head;
  const uint32_t avail = free64 <= 0 ? 0u : free64 < (int64_t)cap ? (uint32_t)free64 : cap;
  const uint32_t h0 = (uint32_t)((uint64_t)head % cap), t0 = (uint32_t)((uint64_t)tail % cap);
  uint32_t wants = 0, gone = 0, all_wants, all_gone, live;
  int from = -1;
  if (tid < R && q.part) {
    from = fork_page(G, q, q.whole);
    wants = from >= 0 && ((s_whole[from / 32] >> (from % 32) & 1) || s_first[from] != R - tid);
  }
  uint32_t at = fork_scan(wants, s_sum, all_wants);
  const bool copied = wants && at < avail, refused = wants && !copied;
  if (tid < R) {
    const uint32_t c = h0 + at;
    const int last = copied ? ldg(A.ring + (c < cap ? c : c - cap)) : refused ? -1 : -2;  // (-2: the parent's)
    s_last[tid] = last;
    A.src[tid] = copied ? from : -1;
    A.dst[tid] = copied ? last : -1;
    A.n[tid] = copied ? (int32_t)q.part : 0;
    A.seq_len[tid] = (int32_t)(refused ? q.n - q.part : q.n);
  }
  fork_scan(tid < R && (refused ? q.whole : q.n) > 0, s_sum, live);
  bool goes[8];
  const uint32_t p0 = tid * 8;
  const uint32_t freed = s_before[p0 / 32] & ~s_whole[p0 / 32];
#pragma unroll
  for (int i = 0; i < 8; ++i) gone += goes[i] = (freed >> ((p0 + i) % 32) & 1) && s_first[p0 + i] == 0;
  at = fork_scan(gone, s_sum, all_gone);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (goes[i]) {
      const uint32_t c = t0 + at;
      if (at < cap) A.ring[c < cap ? c : c - cap] = (int32_t)(p0 + i);  // (no more than the ring holds)
      ++at;
    }
  if (tid == 0) {
    const uint32_t taken = min(all_wants, avail);
    A.cursor_out[0] = head + taken;
    A.cursor_out[1] = tail + all_gone;
    A.counts[0] = (int32_t)live;
    A.counts[1] = (int32_t)taken;
    A.counts[2] = (int32_t)(all_wants - taken);
    A.counts[3] = (int32_t)all_gone;
  }
  for (int r = w; r < R; r += FORK_THREADS / 64) {
    const ForkReq o = fork_req(G, s_parent[r], s_n[r]);
    const int last = s_last[r];
    for (uint32_t c = lane; c < (uint32_t)A.table_width; c += 64)
      A.table_out[(int64_t)r * A.table_out_stride + c] = last != -2 && c == o.whole ? last : fork_page(G, o, c);
  }
}

// ---------------------------------------------------------------------------
// copies of pages, positions moved together
// ---------------------------------------------------------------------------

struct MoveArgs {
  char *k, *v;
  int64_t page_stride, token_stride, head_stride, n_pages;  // bytes
  int32_t page_size, n_heads, pieces;                       // 16-byte pieces of a head's row
  const int32_t *src, *dst, *n;
  // compact
  const int32_t *table, *start, *kept, *n_kept;
  int32_t* new_len;
  int64_t table_stride, kept_stride;
  int32_t n_requests, table_width, kept_width, reach;
  uint32_t mul, shift;
};

__device__ __forceinline__ u32x4 ld_piece(const char* p) { return *(const GLOBAL u32x4*)p; }
__device__ __forceinline__ void st_piece(char* p, u32x4 v) { *(GLOBAL u32x4*)p = v; }

// A copy's pieces over the work-groups of a row of the grid, in the cache's
// order, four loads in flight a thread.
__global__ __launch_bounds__(256) void k_cache_copy(MoveArgs A, int n_copies) {
  for (int i = blockIdx.y; i < n_copies; i += gridDim.y) {
    const int s = ldg(A.src + i), d = ldg(A.dst + i), n = min(ldg(A.n + i), A.page_size);
    if (s < 0 || d < 0 || s >= A.n_pages || d >= A.n_pages || s == d || n <= 0) continue;
    const int row = A.n_heads * A.pieces;
    const int64_t all = 2 * (int64_t)n * row, from = s * A.page_stride, to = d * A.page_stride;
    for (int64_t u0 = blockIdx.x * 1024 + threadIdx.x; u0 < all; u0 += gridDim.x * 1024) {
      u32x4 x[4];
      char* at[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t u = min(u0 + 256 * j, all - 1);
        const int64_t t = u / row;
        const int e = (int)(u - t * row), h = e / A.pieces;
        char* base = t < n ? A.k : A.v;
        const int64_t off = (t < n ? t : t - n) * A.token_stride + h * A.head_stride + 16 * (e - h * A.pieces);
        x[j] = ld_piece(base + from + off);
        at[j] = base + to + off;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (u0 + 256 * j < all) st_piece(at[j], x[j]);
    }
  }
}

// A wave moves one request's column of LP 16-byte pieces of one head of K or of
// V, 16 loads a trip. A position only moves down, so what a later trip reads is
// not what an earlier one writes: a trip's loads are asked for before the last
// one's stores, which wait for all of their own trip's loads. Which positions move
// is known three trips ahead, their pages two.
template <int LP>
__global__ __launch_bounds__(64) void k_cache_compact(MoveArgs A) {
  constexpr int U = 16, ROWS = 64 / LP, TRIP = U * ROWS, PL = TRIP / 64;  // positions of a load, of a trip, of a trip a lane
  const int lane = threadIdx.x, cols = (A.pieces + LP - 1) / LP;
  const int64_t per = 2ll * A.n_heads * cols, units = per * A.n_requests;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int r = (int)(unit / per);
    const int x = (int)(unit - r * per), col = x % cols, h = x / cols % A.n_heads;
    char* base = (x / cols < A.n_heads ? A.k : A.v) + h * A.head_stride;
    const int piece = col * LP + lane % LP;
    const bool mine = piece < A.pieces;
    base += 16 * (mine ? piece : 0);
    const uint32_t a = (uint32_t)max(ldg(A.start + r), 0);
    const int n = min(max(ldg(A.n_kept + r), 0), A.kept_width);
    if (A.new_len && x == 0 && lane == 0) A.new_len[r] = (int32_t)min(a + (uint32_t)n, 1u << 30);
    const int32_t *tab = A.table + r * A.table_stride, *kept = A.kept + r * A.kept_stride;
    const auto column = [&](uint32_t t) { return (uint32_t)(((uint64_t)t * A.mul) >> (31 + A.shift)); };
    struct Moves {  // of a trip, PL positions a lane: where from (-1: it stays), and the two pages
      int32_t from[PL], page_from[PL], page_to[PL];
    };
    const auto listed = [&](int i, Moves& m) {
#pragma unroll
      for (int k = 0; k < PL; ++k) {
        const int j = i * TRIP + 64 * k + lane;
        m.from[k] = ldg(kept + min(j, n - 1));
        if (j >= n) m.from[k] = -1;
      }
    };
    const auto look_up = [&](int i, Moves& m) {
#pragma unroll
      for (int k = 0; k < PL; ++k) {
        const uint32_t to = a + (uint32_t)(i * TRIP + 64 * k + lane);
        const bool moves = m.from[k] >= 0 && (uint32_t)m.from[k] > to && m.from[k] < A.reach;  // (so `to` is in reach too)
        if (!moves) m.from[k] = -1;
        m.page_from[k] = ldg(tab + (moves ? column((uint32_t)m.from[k]) : 0));
        m.page_to[k] = ldg(tab + (moves ? column(to) : 0));
      }
    };
    const int trips = (n + TRIP - 1) / TRIP;
    if (trips == 0) continue;
    Moves m0, m1, m2;  // of this trip, and the next two
    listed(0, m0);
    listed(1, m1);
    look_up(0, m0);
    u32x4 old[U];
    int64_t old_to[PL];
#pragma unroll
    for (int k = 0; k < PL; ++k) old_to[k] = -1;
    const auto store = [&]() {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t t = __shfl(old_to[u * ROWS / 64], u * ROWS % 64 + lane / LP, 64);
        if (t >= 0 && mine) st_piece(base + t, old[u]);
      }
    };
    for (int i = 0; i < trips; ++i) {
      listed(i + 2, m2);
      look_up(i + 1, m1);
      int64_t from[PL], to[PL];
#pragma unroll
      for (int k = 0; k < PL; ++k) {
        const uint32_t s = (uint32_t)m0.from[k], d = a + (uint32_t)(i * TRIP + 64 * k + lane);
        const bool go = m0.from[k] >= 0 && (uint32_t)m0.page_from[k] < (uint64_t)A.n_pages && (uint32_t)m0.page_to[k] < (uint64_t)A.n_pages;
        from[k] = go ? m0.page_from[k] * A.page_stride + (int64_t)(s - column(s) * A.page_size) * A.token_stride : 0;
        to[k] = go ? m0.page_to[k] * A.page_stride + (int64_t)(d - column(d) * A.page_size) * A.token_stride : -1;
      }
      u32x4 v[U];  // (of a position that stays: some other, so that the loads can be counted)
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = ld_piece(base + __shfl(from[u * ROWS / 64], u * ROWS % 64 + lane / LP, 64));
      // the last trip's loads are done when these 16 are the only operations out
      asm volatile("s_waitcnt vmcnt(16)" ::: "memory");
      store();
#pragma unroll
      for (int u = 0; u < U; ++u) old[u] = v[u];
#pragma unroll
      for (int k = 0; k < PL; ++k) old_to[k] = to[k];
      m0 = m1, m1 = m2;
    }
    wait_vm_all();
    store();
  }
}

// Waves from which on a compaction's columns are 256 bytes, and from which on 128 (a
// line of the L2); with fewer they are 64, or 32 where those are below the last, so
// that more waves each make fewer trips.
// Half of r x 16000 positions of 8 heads of 256 bytes, times in a graph: r = 16, 256
// waves of 256 bytes 280 us, 512 of 128 204, 1024 of 64 252; r = 8, 128 bytes 177, 64
// 192; r = 4, 151 and 120, of 32 161; r = 1, 130, 87 and 72; 8 x 9304 of one head of 128
// bytes, of 64 58, of 32 45 (lists of up to 2000: equal). 1024
// waves of 256, trees of 24 tokens of 64 requests, 5.2 us of the kernel, of 128 6.8.
// (Bound by the memory where waves are many: r = 16, 787 MB, 4.1 TB/s.)
constexpr int64_t COMPACT_WAVES = 1024, COMPACT_FEW = 256, COMPACT_FEWER = 144;

// The workspace of a fork. What a call leaves behind comes first, with room for the
// most requests and pages, and the marks, which are zero between calls, behind it:
// calls of any sizes may use one workspace in turn.
constexpr int64_t FORK_MOST = 65536, FORK_MOST_PAGES = 1 << 24;
struct Parts {
  int64_t need, need_sum, free_sum, first, whole, before, bytes;
};
Parts fork_parts(int64_t n_pages) {
  const auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  Parts p;
  p.need = 0;
  p.need_sum = p.need + 4 * FORK_MOST;
  p.free_sum = p.need_sum + 4 * FORK_MOST / FORK_THREADS;
  p.first = p.free_sum + 4 * FORK_MOST_PAGES / FORK_PAGES;
  p.whole = p.first + up(4 * n_pages);
  p.before = p.whole + up(n_pages);
  p.bytes = p.before + up(n_pages);
  return p;
}

struct Range {
  const void* p;
  int64_t bytes;
};
bool meet(const Range& a, const Range& b) { return a.bytes > 0 && b.bytes > 0 && rows_meet(a.p, 0, a.bytes, b.p, 0, b.bytes, 1); }

// x / d for 0 <= x < 2^31: multiply by ceil(2^(31 + shift) / d)
void division(int32_t d, uint32_t& mul, uint32_t& shift) {
  shift = 0;
  while ((1 << shift) < d) ++shift;
  mul = (uint32_t)((((uint64_t)1 << (31 + shift)) + d - 1) / d);
}

MoveArgs move_args(const scute_kv_cache* C) {
  MoveArgs A{};
  const int64_t es = C->dtype == SCUTE_F32 ? 4 : 2;
  A.k = (char*)C->k, A.v = (char*)C->v;
  A.page_stride = C->page_stride * es, A.token_stride = C->token_stride * es, A.head_stride = C->head_stride * es;
  A.n_pages = C->n_pages, A.page_size = C->page_size, A.n_heads = C->n_kv_heads;
  A.pieces = (int)(C->head_dim * es / 16);
  return A;
}

scute_status done(const char* fn) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SCUTE_OK : hip_fail(e, fn);
}

}  // namespace scute

using namespace scute;

extern "C" scute_status scute_cache_fork_workspace(int32_t n_requests, int32_t n_pages, int64_t* bytes) {
  if (!bytes) return fail(SCUTE_E_INVALID, "scute_cache_fork_workspace: bytes is null");
  if (n_requests < 0 || n_requests > FORK_MOST || n_pages < 1 || n_pages > FORK_MOST_PAGES)
    return fail(SCUTE_E_SHAPE, "scute_cache_fork_workspace: n_requests must be in [0, 65536] and n_pages in [1, 2^24]");
  *bytes = fork_parts(n_pages).bytes;
  return SCUTE_OK;
}

extern "C" scute_status scute_cache_fork(const scute_cache_fork_args* A, void* stream) {
  const char* fn = "scute_cache_fork";
  if (!A) return fail(SCUTE_E_INVALID, "scute_cache_fork: args is null");
  if (A->device < 0) return fail(SCUTE_E_INVALID, "scute_cache_fork: device must be >= 0");
  if (A->n_requests < 0 || A->n_requests > FORK_MOST)
    return fail(SCUTE_E_SHAPE, "scute_cache_fork: n_requests must be in [0, 65536]");
  if (A->page_size < 1 || A->page_size > 65536)
    return fail(SCUTE_E_SHAPE, "scute_cache_fork: page_size must be in [1, 65536]");
  const int64_t big = (int64_t)1 << 40;
  if (A->table_width < 1 || A->table_width > (1 << 24) || A->table_stride < A->table_width || A->table_stride > big ||
      A->table_out_stride < A->table_width || A->table_out_stride > big)
    return fail(SCUTE_E_SHAPE, "scute_cache_fork: table_width must be in [1, 2^24] and at most the tables' strides");
  if (A->ring_size < 1 || A->ring_size > (1 << 30))
    return fail(SCUTE_E_SHAPE, "scute_cache_fork: ring_size must be in [1, 2^30]");
  if (A->n_pages < 1 || A->n_pages > FORK_MOST_PAGES)
    return fail(SCUTE_E_SHAPE, "scute_cache_fork: n_pages must be in [1, 2^24]");
  if (A->window < 0 || A->sinks < 0) return fail(SCUTE_E_SHAPE, "scute_cache_fork: window and sinks must be >= 0");
  const bool some = A->n_requests > 0;
  if (!A->ring || !A->cursor || !A->cursor_out || !A->counts || !A->workspace ||
      (some && (!A->len || !A->parent || !A->table || !A->table_out || !A->seq_len || !A->src || !A->dst || !A->n)))
    return fail(SCUTE_E_INVALID, "scute_cache_fork: null pointer");
  for (const void* p : {(const void*)A->len, (const void*)A->parent, (const void*)A->keep, (const void*)A->table,
                        (const void*)A->ring, (const void*)A->table_out, (const void*)A->seq_len, (const void*)A->src,
                        (const void*)A->dst, (const void*)A->n, (const void*)A->counts})
    if ((uintptr_t)p & 3) return fail(SCUTE_E_INVALID, "scute_cache_fork: misaligned pointer");
  if (((uintptr_t)A->cursor | (uintptr_t)A->cursor_out) & 7)
    return fail(SCUTE_E_INVALID, "scute_cache_fork: misaligned pointer");
  if ((uintptr_t)A->workspace & 255) return fail(SCUTE_E_INVALID, "scute_cache_fork: workspace must be 256-byte aligned");
  const int64_t R = A->n_requests;
  const Parts P = fork_parts(A->n_pages);
  if (A->workspace_bytes < P.bytes) return fail(SCUTE_E_INVALID, "scute_cache_fork: the workspace is too small");
  // work-groups read the inputs while others write the outputs
  const int64_t extent = some ? 4 * ((R - 1) * A->table_stride + A->table_width) : 0;
  const int64_t extent_out = some ? 4 * ((R - 1) * A->table_out_stride + A->table_width) : 0;
  const Range ins[] = {{A->cursor, 16}, {A->len, 4 * R}, {A->parent, 4 * R}, {A->keep, A->keep ? 4 * R : 0}, {A->table, extent}};
  const Range outs[] = {{A->cursor_out, 16}, {A->counts, 16}, {A->ring, 4 * (int64_t)A->ring_size},
                        {A->table_out, extent_out}, {A->seq_len, 4 * R}, {A->src, 4 * R}, {A->dst, 4 * R}, {A->n, 4 * R},
                        {A->workspace, P.bytes}};
  for (const Range& o : outs) {
    for (const Range& i : ins)
      if (meet(o, i)) return fail(SCUTE_E_INVALID, "scute_cache_fork: an output is also an input");
    for (const Range* b = outs; b < &o; ++b)
      if (meet(o, *b)) return fail(SCUTE_E_INVALID, "scute_cache_fork: outputs overlap");
  }
  OnDevice g(A->device);
  if (!g.ok()) return hip_fail(g.err, fn);
  char* ws = (char*)A->workspace;
  ForkArgs G{};
  G.a = *A;
  division(A->page_size, G.mul, G.shift);
  G.first = (int32_t*)(ws + P.first);
  G.whole = (uint8_t*)(ws + P.whole), G.before = (uint8_t*)(ws + P.before);
  G.need = (uint32_t*)(ws + P.need);
  G.need_sum = (uint32_t*)(ws + P.need_sum), G.free_sum = (uint32_t*)(ws + P.free_sum);
  G.req_blocks = (int)((R + FORK_THREADS - 1) / FORK_THREADS);
  G.page_blocks = (A->n_pages + FORK_PAGES - 1) / FORK_PAGES;
  const hipStream_t s = (hipStream_t)stream;
  if (A->n_pages <= FORK_ONE_PAGES && R * ((A->table_width + 63) / 64) <= FORK_ONE_PIECES) {
    hipLaunchKernelGGL(k_fork_one, dim3(1), dim3(FORK_THREADS), 0, s, G);
    return done(fn);
  }
  // several work-groups a row where the rows are few
  const int64_t rows = std::min<int64_t>(R, 4096);
  const auto parts = [&](int64_t each) {
    return std::max<int64_t>(1, std::min<int64_t>((A->table_width + each - 1) / each, 2048 / std::max<int64_t>(rows, 1)));
  };
  if (some)
    hipLaunchKernelGGL(k_fork_mark, dim3((unsigned)parts(256), (unsigned)rows), dim3(256), 0, s, G);
  hipLaunchKernelGGL(k_fork_sums, dim3((unsigned)(G.page_blocks + G.req_blocks)), dim3(FORK_THREADS), 0, s, G);
  G.row_parts = (int)parts(FORK_THREADS);
  hipLaunchKernelGGL(k_fork_apply, dim3((unsigned)(G.page_blocks + 1 + rows * G.row_parts)), dim3(FORK_THREADS), 0, s, G);
  return done(fn);
}

extern "C" scute_status scute_cache_copy(const scute_kv_cache* C, const int32_t* src, const int32_t* dst,
                                         const int32_t* n, int32_t n_copies, void* stream) {
  const char* fn = "scute_cache_copy";
  scute_status st = check_cache(C, fn);
  if (st != SCUTE_OK) return st;
  if (n_copies < 0 || n_copies > (1 << 20)) return fail(SCUTE_E_SHAPE, "scute_cache_copy: n_copies must be in [0, 2^20]");
  if (n_copies == 0) return SCUTE_OK;
  if (!src || !dst || !n) return fail(SCUTE_E_INVALID, "scute_cache_copy: null pointer");
  if (((uintptr_t)src | (uintptr_t)dst | (uintptr_t)n) & 3)
    return fail(SCUTE_E_INVALID, "scute_cache_copy: misaligned pointer");
  OnDevice g(C->device);
  if (!g.ok()) return hip_fail(g.err, fn);
  MoveArgs A = move_args(C);
  A.src = src, A.dst = dst, A.n = n;
  const int64_t all = 2ll * C->page_size * A.n_heads * A.pieces, rows = std::min<int64_t>(n_copies, 4096);
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>((all + 1023) / 1024, 8192 / rows));
  hipLaunchKernelGGL(k_cache_copy, dim3((unsigned)parts, (unsigned)rows), dim3(256), 0, (hipStream_t)stream, A, n_copies);
  return done(fn);
}

extern "C" scute_status scute_cache_compact(const scute_kv_cache* C, const int32_t* table, int64_t table_stride,
                                            int32_t n_requests, int32_t table_width, const int32_t* start,
                                            const int32_t* kept, int64_t kept_stride, int32_t kept_width,
                                            const int32_t* n_kept, int32_t* new_len, void* stream) {
  const char* fn = "scute_cache_compact";
  scute_status st = check_cache(C, fn);
  if (st != SCUTE_OK) return st;
  const int64_t big = (int64_t)1 << 40;
  if (n_requests < 0 || n_requests > 65536)
    return fail(SCUTE_E_SHAPE, "scute_cache_compact: n_requests must be in [0, 65536]");
  if (table_width < 1 || table_width > (1 << 24) || table_stride < table_width || table_stride > big)
    return fail(SCUTE_E_SHAPE, "scute_cache_compact: table_width must be in [1, 2^24] and at most table_stride");
  if (kept_width < 0 || kept_width > (1 << 29) || kept_stride < kept_width || kept_stride > big)
    return fail(SCUTE_E_SHAPE, "scute_cache_compact: kept_width must be in [0, 2^29] and at most kept_stride");
  if (n_requests == 0) return SCUTE_OK;
  if (!table || !start || (!kept && kept_width) || !n_kept) return fail(SCUTE_E_INVALID, "scute_cache_compact: null pointer");
  if (((uintptr_t)table | (uintptr_t)start | (uintptr_t)kept | (uintptr_t)n_kept | (uintptr_t)new_len) & 3)
    return fail(SCUTE_E_INVALID, "scute_cache_compact: misaligned pointer");
  const int64_t R = n_requests;
  const Range out{new_len, new_len ? 4 * R : 0};
  for (const Range& i : {Range{start, 4 * R}, Range{n_kept, 4 * R}, Range{table, 4 * ((R - 1) * table_stride + table_width)},
                         Range{kept, kept_width ? 4 * ((R - 1) * kept_stride + kept_width) : 0}})
    if (meet(out, i)) return fail(SCUTE_E_INVALID, "scute_cache_compact: new_len is also an input");
  OnDevice g(C->device);
  if (!g.ok()) return hip_fail(g.err, fn);
  MoveArgs A = move_args(C);
  A.table = table, A.table_stride = table_stride, A.table_width = table_width;
  A.start = start, A.kept = kept, A.kept_stride = kept_stride, A.kept_width = kept_width, A.n_kept = n_kept;
  A.new_len = new_len, A.n_requests = n_requests;
  A.reach = (int32_t)std::min<int64_t>((int64_t)table_width * C->page_size, (int64_t)1 << 30);
  division(C->page_size, A.mul, A.shift);
  const int64_t columns = 2 * R * A.n_heads, most = 1 << 22;
  const hipStream_t s = (hipStream_t)stream;
  const auto blocks = [&](int lp) { return dim3((unsigned)std::min(most, columns * ((A.pieces + lp - 1) / lp))); };
  if (columns * ((A.pieces + 15) / 16) >= COMPACT_WAVES)
    hipLaunchKernelGGL(k_cache_compact<16>, blocks(16), dim3(64), 0, s, A);
  else if (columns * ((A.pieces + 7) / 8) >= COMPACT_FEW)
    hipLaunchKernelGGL(k_cache_compact<8>, blocks(8), dim3(64), 0, s, A);
  else if (columns * ((A.pieces + 3) / 4) >= COMPACT_FEWER)
    hipLaunchKernelGGL(k_cache_compact<4>, blocks(4), dim3(64), 0, s, A);
  else
    hipLaunchKernelGGL(k_cache_compact<2>, blocks(2), dim3(64), 0, s, A);
  return done(fn);
}
