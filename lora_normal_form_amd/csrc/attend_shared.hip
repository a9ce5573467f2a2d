// Attention of rows whose contexts begin with the same positions
// (scute_shared_attention).

#include <algorithm>

#include "attend.h"
#include "attend_host.h"
#include "shared_cut.h"

namespace scute {

// Where a row's partial results lie.
struct alignas(16) ShRow {
  // shared positions: the row's group has `tiles` wide tiles of columns (row of the
  // group times heads of a key head, and head of it; the row's first is col0) for
  // each key head, the x0-th on, of `units` units from the u0-th on (0: nothing
  // shared)
  int32_t units, tiles, col0;
  uint32_t u0, x0;
  // its own: `own` tiles a head behind `before` of the rows before it, of row
  // `lead`'s run, whose column `at` is the row's first
  int32_t own;
  uint32_t before;
  int32_t lead, at, pad[3];
};
struct ShPlan {
  uint32_t each_shared, each_own;  // units of a gang, tiles of a chunk
  int32_t taken;                   // chunks taken behind the waves' first; 0 between calls
};
static_assert(sizeof(ShPlan) <= ATT_PLAN_BYTES);

struct SharedArgs {
  const void *q, *k, *v;
  void* out;
  const int32_t *table, *len, *req, *group, *shared;
  ShRow* rows;
  ShPlan* plan;
  float *seeds, *own;  // partial results of shared and of own positions
  int64_t q_stride, out_stride, page_stride, token_stride, head_stride, table_stride, n_pages;
  uint32_t ps_mul;
  int32_t n_rows, n_groups, n_kv, heads, head_dim, page_size, ps_shift, reach, n_requests, max_tiles;
  int32_t cw, pw;                       // waves side by side in a work-group's columns, and one after the other in positions
  int32_t gang;                         // work-groups of a wide tile of columns
  int32_t together, q_tiles, own_cols;  // rows of a run at most; query tiles of a key head; columns of an own slot
  int32_t negate;    // the scale is below 0
  float scale_log2;  // its magnitude times log2(e), above 0 (so that what is masked stays at -inf)
};

// Geometry of one instantiation.
constexpr int sh_stage(int es, int dp) {
  return 8192 / (dp * es) > 32 / (es / 2) ? 8192 / (dp * es) : 32 / (es / 2);  // (a tile at least)
}
template <typename T, int DP>
struct ShGeo {
  using G = AttGeo<T, DP>;
  static constexpr int QT = DP * G::ES >= 1024 ? 1 : 2;  // query tiles a wave (one where two would not fit the registers)
  static constexpr int NW = SH_WAVES;                    // waves of a work-group
  static constexpr int WCOLS = 16 * QT;                  // columns of a wave
  static constexpr int ROW = DP * G::ES;                 // bytes of a position in LDS
  static constexpr int STAGE = sh_stage(G::ES, DP);      // positions staged at once: a unit
  static constexpr int BYTES = STAGE * ROW, RING = (DP <= 128 ? 32768 : 65536) / BYTES;  // bytes of a stage of K (of V), stages in LDS
  static constexpr int PIECES = ROW / 16;                // 16-byte pieces of a position
  static constexpr int LOADS = BYTES / 1024 / NW;        // a wave's loads of 1 KB a stage (of K, and of V)
};
// where LDS holds piece p of a stage's position: rows that are read together are
// spread over the banks
template <int ROW>
__device__ __forceinline__ int sh_slot(int row, int p) {
  return ROW >= 256 ? (p & ~15) | ((p ^ row) & 15) : p ^ ((row >> 1) & 7);
}
// Vectors of W dwords from LDS at a[0 .. 3] + O0 (out[0 .. 3]) and, where O1 is not
// 0, + O1 (out[4 .. 7]), there when it returns. In assembly because the compiler
// makes its own reads of LDS wait for every load to LDS that is under way (each
// stage would wait for the three behind it).
template <int W, int O0, int O1>
__device__ __forceinline__ void lds_read(const uint32_t (&a)[4], uint32_t (*const (&out)[8])) {
  typedef uint32_t vec __attribute__((ext_vector_type(W)));
  vec v[8];
  if constexpr (W == 4 && O1 != 0) {
    asm volatile(
        "ds_read_b128 %0, %8 offset:%12\n\tds_read_b128 %1, %9 offset:%12\n\t"
        "ds_read_b128 %2, %10 offset:%12\n\tds_read_b128 %3, %11 offset:%12\n\t"
        "ds_read_b128 %4, %8 offset:%13\n\tds_read_b128 %5, %9 offset:%13\n\t"
        "ds_read_b128 %6, %10 offset:%13\n\tds_read_b128 %7, %11 offset:%13\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "n"(O0), "n"(O1)
        : "memory");
  } else if constexpr (W == 2 && O1 != 0) {
    asm volatile(
        "ds_read_b64 %0, %8 offset:%12\n\tds_read_b64 %1, %9 offset:%12\n\t"
        "ds_read_b64 %2, %10 offset:%12\n\tds_read_b64 %3, %11 offset:%12\n\t"
        "ds_read_b64 %4, %8 offset:%13\n\tds_read_b64 %5, %9 offset:%13\n\t"
        "ds_read_b64 %6, %10 offset:%13\n\tds_read_b64 %7, %11 offset:%13\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "n"(O0), "n"(O1)
        : "memory");
  } else {
    static_assert(W == 4 && O1 == 0);
    asm volatile(
        "ds_read_b128 %0, %4 offset:%8\n\tds_read_b128 %1, %5 offset:%8\n\t"
        "ds_read_b128 %2, %6 offset:%8\n\tds_read_b128 %3, %7 offset:%8\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "n"(O0)
        : "memory");
  }
#pragma unroll
  for (int i = 0; i < (O1 != 0 ? 8 : 4); ++i)
#pragma unroll
    for (int e = 0; e < W; ++e) out[i][e] = v[i][e];
}
__device__ __forceinline__ float max_over_rows(float v) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
  const u32x2 b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b.x), __uint_as_float(b.y));
}

constexpr int64_t SH_SAVED = 256 << 20;  // bytes
constexpr int SH_TILES = 1 << 22;  // (group, key head, tile)s stay below it

struct ShGroup {
  int row, rows, n, tiles, units;  // first row, rows, shared positions, wide tiles of columns, units of positions
};
template <typename S>
__device__ __forceinline__ ShGroup sh_group(const SharedArgs& A, int g) {
  ShGroup q;
  const int a = min(max(ldg(A.group + g), 0), A.n_rows), b = min(max(ldg(A.group + g + 1), 0), A.n_rows);
  q.row = a, q.rows = max(b - a, 0);
  q.n = min(max(ldg(A.shared + g), 0), A.reach);
  const int wide = S::WCOLS * A.cw * A.gang;
  q.tiles = (int)(((int64_t)q.rows * A.heads + wide - 1) / wide);
  q.units = q.tiles ? (q.n + S::STAGE - 1) / S::STAGE : 0;
  return q;
}
__device__ __forceinline__ int sh_len(const SharedArgs& A, int row) {
  const int len = ldg(A.len + row), req = A.req ? ldg(A.req + row) : row;
  return (uint32_t)req < (uint32_t)A.n_requests ? min(max(len, 0), A.reach) : 0;
}

// What a work-group knows of the call's groups and rows: in LDS, for each thread's
// groups and rows.
struct ShShared {
  uint32_t u[257], x[257];   // units and (group, key head, tile)s of the groups before the thread's
  int row[257];              // its groups' first row
  int end[256], n[256];      // the first of its groups: the row behind it, shared positions
  uint32_t t[257];           // tiles a head of the rows before the thread's
  uint32_t sum[2][4];
  unsigned long long lead[8];
};
struct ShCall {
  int per_g, per_r;  // groups and rows a thread
  bool fits;
};

// index of the last border (of 256, the first 0) that is <= x
template <typename B>
__device__ __forceinline__ int sh_find(const B* b, B x) {
  int lo = 0;
#pragma unroll
  for (int step = 128; step > 0; step >>= 1)
    if (b[lo + step] <= x) lo += step;
  return lo;
}
// the group of a row: f(group, units before it, tiles before it); whether it has one
template <typename S, typename F>
__device__ __forceinline__ bool sh_group_of(const SharedArgs& A, const ShCall& c, const ShShared& L, int row, F f) {
  if (!c.fits) return false;
  const int lo = sh_find(L.row, row);
  uint32_t u = L.u[lo], x = L.x[lo];
  for (int g = lo * c.per_g; g < min(A.n_groups, (lo + 1) * c.per_g); ++g) {
    const ShGroup q = sh_group<S>(A, g);
    if (row >= q.row && row < q.row + q.rows) {
      f(q, u, x);
      return true;
    }
    u += (uint32_t)q.units * q.tiles * A.n_kv;
    x += (uint32_t)(q.units ? q.tiles : 0) * A.n_kv;
  }
  return false;
}
// positions that a row shares
template <typename S>
__device__ __forceinline__ int sh_from(const SharedArgs& A, const ShCall& c, const ShShared& L, int row) {
  if (c.per_g == 1) {
    const int lo = sh_find(L.row, row);
    return c.fits && row >= L.row[lo] && row < L.end[lo] ? L.n[lo] : 0;
  }
  int n = 0;
  sh_group_of<S>(A, c, L, row, [&](const ShGroup& q, uint32_t, uint32_t) { n = q.n; });
  return n;
}

// A run: up to `together` rows of one request that follow each other (as many as
// fit 16 columns with all heads of a key head, from multiples of `together` on),
// which are read for together. Its positions lo .. n - 1, those that every row of
// it with any sees every_lo .. every_n - 1.
struct ShRun {
  int row, rows, req, lo, n, every_lo, every_n, tiles;
};
// f(run) for the runs of rows base .. base + together - 1
template <typename S, int TILE, typename F>
__device__ __forceinline__ void sh_runs(const SharedArgs& A, const ShCall& c, const ShShared& L, int base, F f) {
  int q[4], n[4], lo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = min(base + j, A.n_rows - 1);
    n[j] = 0, q[j] = -1;
    if (j < A.together) {
      n[j] = ldg(A.len + row);
      q[j] = A.req ? ldg(A.req + row) : row;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    lo[j] = 0;
    if (j < A.together && base + j < A.n_rows) {
      n[j] = (uint32_t)q[j] < (uint32_t)A.n_requests ? min(max(n[j], 0), A.reach) : 0;
      lo[j] = min(n[j], sh_from<S>(A, c, L, base + j));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= A.together || base + i >= A.n_rows || (i > 0 && q[i] == q[i > 0 ? i - 1 : 0])) continue;
    ShRun r{base + i, 0, q[i], 0x7FFFFFFF, 0, 0, 0x7FFFFFFF, 0};
    bool on = true;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j < i) continue;
      on = on && j < A.together && base + j < A.n_rows && q[j] == q[i];
      if (!on) continue;
      ++r.rows;
      if (n[j] > lo[j]) {
        r.lo = min(r.lo, lo[j]), r.n = max(r.n, n[j]);
        r.every_lo = max(r.every_lo, lo[j]), r.every_n = min(r.every_n, n[j]);
      }
    }
    r.lo = min(r.lo, r.n);
    r.tiles = r.n > r.lo ? (r.n + TILE - 1) / TILE - r.lo / TILE : 0;
    f(r);
  }
}

// The weights of a tile's scores, in their place: the column's sum, and its sums of
// values where the reference of its powers of two moves. It moves where a score
// passes it by 2^8: until then the powers stay far inside fp32, and nothing has to
// cross lanes.
template <typename G>
__device__ __forceinline__ void sh_weights(const SharedArgs& A, f32x4 (&sc)[G::SUB], float& mx, float& l,
                                           f32x4 (&acc)[G::NG][G::VD]) {
  float tm = sc[0][0];
#pragma unroll
  for (int sb = 0; sb < G::SUB; ++sb)
#pragma unroll
    for (int j = 0; j < 4; ++j) tm = fmaxf(tm, sc[sb][j]);
  if (__any(fmaf(tm, A.scale_log2, -mx) > 8.f)) {
    const float mn = fmaxf(mx, max_over_rows(tm) * A.scale_log2);
    const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(mx - mn);
    l *= f;
#pragma unroll
    for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
      for (int e = 0; e < G::VD; ++e) acc[ng][e] *= f;
    mx = mn;
  }
  const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
  for (int sb = 0; sb < G::SUB; ++sb)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sc[sb][j] = __builtin_amdgcn_exp2f(fmaf(sc[sb][j], A.scale_log2, -ref));
      l += sc[sb][j];
    }
}
// waits until at most n vector memory operations are out (n rounded down to what
// there is an instruction for)
__device__ __forceinline__ void sh_wait(int n) {
#define WAIT(x) \
  else if (n >= x) __builtin_amdgcn_s_waitcnt(vmcnt_imm(x))
  if (n >= 16) __builtin_amdgcn_s_waitcnt(vmcnt_imm(16));
  WAIT(12);
  WAIT(10);
  WAIT(8);
  WAIT(6);
  WAIT(4);
  WAIT(2);
  else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
#undef WAIT
}
// Elements of a dword of V that are not finite become 0; whether there are any.
template <int ES>
__device__ __forceinline__ bool sh_finite(uint32_t& v) {
  const bool hi = (v & 0x7F800000u) == 0x7F800000u, lo = ES == 2 && (v & 0x7F80u) == 0x7F80u;
  v = ES == 4 ? (hi ? 0u : v) : (hi ? v & 0xFFFFu : v) & (lo ? 0xFFFF0000u : ~0u);
  return hi || lo;
}
// What is not finite of the elements at p (one load of a lane) to row r of the sums
// of a column that sees it: they are not finite then, whatever the weight.
template <typename G>
__device__ __forceinline__ void sh_add_odd(const char* p, bool seen, f32x4 (&acc)[G::VD], int r) {
  typedef uint32_t vec __attribute__((ext_vector_type(G::VB / 4)));
  const vec x = *(const vec*)p;
#pragma unroll
  for (int i = 0; i < G::VD; ++i) {
    const float v = __uint_as_float(G::ES == 4 ? x[i % (G::VB / 4)] : i & 1 ? x[i / 2] & 0xFFFF0000u : x[i / 2] << 16);
    if (!isfinite(v) && seen) acc[i][r] += v;
  }
}

// Sums of the softmax over a group's shared positions for all its rows: a
// product of tall matrices, so K and V go through LDS once for up to 128 columns
// (rows times the heads of a key head), 32 columns a wave: nothing is joined
// between waves. Where the columns do not fill the waves, the waves of a column
// take stages in turn.
template <typename T, int DP, bool PAGE16, bool EXACT>
__device__ __forceinline__ void sh_prefix(const SharedArgs& A, const ShCall& call, ShShared& L,
                                          char (*s_kv)[2 * ShGeo<T, DP>::BYTES], uint32_t gang, int member,
                                          uint32_t each) {
  using G = AttGeo<T, DP>;
  using S = ShGeo<T, DP>;
  constexpr int TILE = G::TILE, SUB = G::SUB, QT = S::QT, NW = S::NW;
  const int tid = threadIdx.x, lane = tid & 63, w = uni(tid >> 6), m16 = lane & 15, gq = lane >> 4;
  const int D = EXACT ? DP : A.head_dim, row_bytes = D * G::ES;
  const int COLS = S::WCOLS * A.cw, pw = A.pw, wc = w % A.cw, wp = w / A.cw;  // the wave's columns and turn
  const uint32_t total = L.u[256];
  const uint32_t u_end = (uint32_t)min((uint64_t)total, (uint64_t)(gang + 1) * each);
  for (uint32_t u = (uint32_t)min((uint64_t)total, (uint64_t)gang * each); u < u_end;) {
    const int lo = sh_find(L.u, u);
    uint32_t u0 = L.u[lo], x = L.x[lo];
    ShGroup q{};
    for (int g = lo * call.per_g; g < A.n_groups; ++g) {  // (the next border is past u)
      q = sh_group<S>(A, g);
      const uint32_t n = (uint32_t)q.units * q.tiles * A.n_kv;
      if (u - u0 < n) break;
      u0 += n, x += (uint32_t)(q.units ? q.tiles : 0) * A.n_kv;
    }
    q = {uni(q.row), uni(q.rows), uni(q.n), uni(q.tiles), uni(q.units)};
    u0 = (uint32_t)uni((int)u0), x = (uint32_t)uni((int)x);
    if (q.units == 0) return;  // (only if the lengths change while the call runs)
    const uint32_t i = (u - u0) / in_place(q.units);
    const int kvh = i / in_place(q.tiles), ct = (i - kvh * q.tiles) * A.gang + member, first = u - u0 - i * q.units;
    const int last = min((uint32_t)q.units, first + (u_end - u));  // units first .. last - 1 of the group's
    x += i;
    u += last - first;

    // the row that sees most of the shared positions, the first of those: its pages are read
    unsigned long long best = 0;
    for (int r = tid; r < q.rows; r += 64 * NW) {
      const unsigned long long v = (unsigned long long)min(sh_len(A, q.row + r), q.n) << 32 | (0xFFFFFFFFu - (uint32_t)r);
      best = v > best ? v : best;
    }
    for (int o = 32; o > 0; o >>= 1) {
      const unsigned long long v = __shfl_xor(best, o, 64);
      best = v > best ? v : best;
    }
    __syncthreads();  // (the previous piece is done with LDS)
    if (lane == 0) L.lead[w] = best;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NW; ++k) best = L.lead[k] > best ? L.lead[k] : best;
    const int reach = uni((int)(best >> 32));  // positions that some row sees
    const int lead = q.row + uni((int)(0xFFFFFFFFu - (uint32_t)best));
    const int units = min(last, (reach + S::STAGE - 1) / S::STAGE) - first;

    // this lane's columns
    int my_n[QT];
    uint4 qf[QT][G::NC];
    int n_min = 0x7FFFFFFF, n_max = 0;
#pragma unroll
    for (int y = 0; y < QT; ++y) {
      const int c = ct * COLS + (wc * QT + y) * 16 + m16, r = c / A.heads, h = kvh * A.heads + (c - r * A.heads);
      my_n[y] = r < q.rows ? min(sh_len(A, q.row + r), q.n) : 0;
      const char* qp = (const char*)A.q + ((int64_t)(q.row + (r < q.rows ? r : 0)) * A.q_stride + (int64_t)h * D) * G::ES;
#pragma unroll
      for (int k = 0; k < G::NC; ++k) {
        const int at = 64 * k + 16 * gq;
        const uint4 v = ldg_b16<false>(qp, EXACT ? at : min(at, row_bytes - 16));
        const uint32_t s = A.negate ? (G::ES == 2 ? 0x80008000u : 0x80000000u) : 0u;  // (a scale below 0 turns q's sign)
        qf[y][k] = my_n[y] > 0 && (EXACT || at < row_bytes) ? make_uint4(v.x ^ s, v.y ^ s, v.z ^ s, v.w ^ s) : make_uint4(0, 0, 0, 0);
      }
      if (my_n[y] > 0) n_min = min(n_min, my_n[y]), n_max = max(n_max, my_n[y]);
    }
    for (int o = 8; o > 0; o >>= 1) {
      n_min = min(n_min, __shfl_xor(n_min, o, 64));
      n_max = max(n_max, __shfl_xor(n_max, o, 64));
    }
    n_min = uni(n_min), n_max = uni(n_max);  // (n_max 0: the wave has no columns that see anything)

    float mx[QT], l[QT];
    f32x4 acc[QT][G::NG][G::VD];
#pragma unroll
    for (int y = 0; y < QT; ++y) {
      mx[y] = -INFINITY, l[y] = 0.f;
#pragma unroll
      for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
        for (int e = 0; e < G::VD; ++e) acc[y][ng][e] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // ---- staging: loads of 1 KB straight to LDS, a step (pw stages) a time,
    // `ahead` steps before it is used ----
    constexpr int ROWS = 1024 / S::ROW;                  // positions of a load
    constexpr int NB = S::STAGE / 16, REACH = 64 / NB;   // blocks of 16 positions of a stage; stages of 64 blocks
    const int steps = (units + pw - 1) / pw, ahead = S::RING / pw - 1;
    const int32_t* tab = A.table + (int64_t)(reach > 0 ? uni(A.req ? ldg(A.req + lead) : lead) : 0) * A.table_stride;
    const int64_t head = (int64_t)kvh * A.head_stride * G::ES;
    const uint32_t tok = (uint32_t)A.token_stride * G::ES;
    const auto page_of = [&](int t) { return (int)(((uint64_t)(uint32_t)t * A.ps_mul) >> (31 + A.ps_shift)); };
    const auto row0 = [&](int j) { return (w + NW * j) * ROWS; };  // the first row of load j
    const auto to_lds = [&](const char* k, const char* v, int s, int j) {
      char* to = s_kv[s % S::RING] + (w + NW * j) * 1024;
      __builtin_amdgcn_global_load_lds((const GLOBAL void*)k, (lds_void*)to, 16, 0, 0);
      __builtin_amdgcn_global_load_lds((const GLOBAL void*)v, (lds_void*)(to + S::BYTES), 16, 0, 0);
    };
    // pages of multiples of 16 positions: where 64 blocks lie, one a lane, and the
    // pages of the next 64; otherwise the pages of a stage's positions, one a lane,
    // of the two stages that are loaded next
    int32_t place_lo = 0, place_hi = 0, raw = 0, raw2 = 0;
    uint64_t bad[2] = {0, 0};                           // blocks on no page, by turns of 64
    uint64_t gone_at[PAGE16 ? 1 : S::RING] = {};        // positions on no page, of stages s, s + 1, ...
    const auto block = [&](int g) { return 16 * min(first * NB + 64 * g + lane, (reach - 1) >> 4); };
    const auto position = [&](int s) { return min((first + min(s, units - 1)) * S::STAGE + lane % S::STAGE, reach - 1); };
    const auto refill = [&](int g) {
      const int t = block(g), at = page_of(t);
      const bool ok = raw >= 0 && raw < A.n_pages;
      const int64_t off = ((int64_t)raw * A.page_stride + (int64_t)(t - at * A.page_size) * A.token_stride) * G::ES + head;
      place_lo = ok ? (int32_t)(uint32_t)off : (int32_t)(uint32_t)head, place_hi = ok ? (int32_t)(off >> 32) : (int32_t)(head >> 32);
      const uint64_t no = __ballot(!ok);
      if (g & 1) bad[1] = no;
      else bad[0] = no;
      raw = ldg(tab + page_of(block(g + 1)));
    };
    const auto load = [&](int s) {  // stage s, or the last again behind it
      if constexpr (PAGE16) {
        if (s % REACH == 0) refill(s / REACH);
#pragma unroll
        for (int j = 0; j < S::LOADS; ++j) {
          const int r = row0(j), b = s % REACH * NB + r / 16;
          const int64_t base = (int64_t)((uint64_t)(uint32_t)lane_of(place_hi, b) << 32 | (uint32_t)lane_of(place_lo, b));
          const int in = r % 16 + lane / S::PIECES, at = 16 * sh_slot<S::ROW>(r + lane / S::PIECES, lane % S::PIECES);
          const uint32_t off = in * tok + (EXACT ? at : min(at, row_bytes - 16));
          to_lds((const char*)A.k + base + off, (const char*)A.v + base + off, s, j);
        }
      } else {
        const int t = position(s);
        const bool ok = raw >= 0 && raw < A.n_pages;
        const int64_t off =
            (ok ? (int64_t)raw * A.page_stride + (int64_t)(t - page_of(t) * A.page_size) * A.token_stride : 0) * G::ES + head;
        raw = raw2;
        raw2 = ldg(tab + page_of(position(s + 2)));
#pragma unroll
        for (int j = 0; j < S::LOADS; ++j) {
          const int r = row0(j) + lane / S::PIECES, at = 16 * sh_slot<S::ROW>(r, lane % S::PIECES);
          const uint32_t lo = __shfl((int)(uint32_t)off, r, 64), hi = __shfl((int)(off >> 32), r, 64);
          const int64_t o = (int64_t)((uint64_t)hi << 32 | lo) + (EXACT ? at : min(at, row_bytes - 16));
          to_lds((const char*)A.k + o, (const char*)A.v + o, s, j);
        }
        gone_at[S::RING - 1] = __ballot(!ok);
      }
    };
    if (units > 0) {
      raw = ldg(tab + page_of(PAGE16 ? block(0) : position(0)));
      if constexpr (!PAGE16) raw2 = ldg(tab + page_of(position(1)));
      if constexpr (PAGE16) {
        for (int s = 0; s < min(ahead, steps) * pw; ++s) load(s);
      } else {
#pragma unroll
        for (int s = 0; s < S::RING - 1; ++s)  // (pw is 1)
          if (s < steps) {
            load(s);
            gone_at[s] = gone_at[S::RING - 1];
          }
      }
    }
    const uint32_t lds = (uint32_t)(uintptr_t)(lds_void*)&s_kv[0][0];
    const uint32_t k_at = m16 * S::ROW + 16 * sh_slot<S::ROW>(m16, gq);  // (chunk c: ^ 64 c, 16 positions on: + 16 ROW)
    uint32_t v_at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 4 * gq + j, b = m16 * G::VB;
      v_at[j] = S::BYTES + row * S::ROW + 16 * sh_slot<S::ROW>(row, b / 16) + b % 16;
    }
    for (int i = 0; i < steps; ++i) {
      // this wave's part of step i is there when those of the steps behind it are the
      // only loads that are out; then all waves' parts are
      sh_wait(min(steps - 1 - i, ahead - 1) * pw * 2 * S::LOADS);
      lds_barrier();
      const int s = i * pw + wp;  // the wave's stage of the step
      uint64_t gone_s = 0;
      if constexpr (PAGE16) {
        const uint64_t b = (s / REACH & 1 ? bad[1] : bad[0]) >> (s % REACH * NB);
#pragma unroll
        for (int x = 0; x < NB; ++x) gone_s |= b >> x & 1 ? 0xFFFFull << (16 * x) : 0ull;
      } else {
        gone_s = gone_at[0];
#pragma unroll
        for (int x = 0; x + 1 < S::RING; ++x) gone_at[x] = gone_at[x + 1];
      }
      const auto next = [&]() {
        if (i + ahead < steps) {
          for (int x = 0; x < pw; ++x) load((i + ahead) * pw + x);
          if constexpr (!PAGE16) gone_at[S::RING - 2] = gone_at[S::RING - 1];
        }
      };
      if (s >= units || (first + s) * S::STAGE >= n_max) {  // (no column of the wave sees any of it)
        next();
        continue;
      }
#pragma unroll 1
      for (int tt = 0; tt < S::STAGE / TILE; ++tt) {
        const int t = (first + s) * S::STAGE + tt * TILE;
        if (tt > 0 && t >= n_max) break;
        AttTile<T, DP, EXACT> tile;
        const uint32_t base = lds + (s % S::RING) * 2 * S::BYTES + tt * TILE * S::ROW;
        if constexpr (G::NC == 2) {  // (two chunks of 32 positions, as four rows)
          static_assert(SUB == 2);
          const uint32_t a[4] = {base + k_at, base + (k_at ^ 64), base + k_at + 16 * S::ROW, base + (k_at ^ 64) + 16 * S::ROW};
          uint32_t* const o[8] = {&tile.k[0][0].x, &tile.k[0][1].x, &tile.k[1][0].x, &tile.k[1][1].x};
          lds_read<4, 0, 0>(a, o);
        } else {
#pragma unroll
          for (int c = 0; c < G::NC; c += 4) {
            const uint32_t a[4] = {base + (k_at ^ (64 * c)), base + (k_at ^ (64 * c + 64)), base + (k_at ^ (64 * c + 128)),
                                   base + (k_at ^ (64 * c + 192))};
            uint32_t* const o[8] = {&tile.k[0][c].x, &tile.k[0][c + 1].x, &tile.k[0][c + 2].x, &tile.k[0][c + 3].x,
                                    &tile.k[SUB - 1][c].x, &tile.k[SUB - 1][c + 1].x, &tile.k[SUB - 1][c + 2].x,
                                    &tile.k[SUB - 1][c + 3].x};
            lds_read<4, 0, SUB == 2 ? 16 * S::ROW : 0>(a, o);
          }
        }
        f32x4 sc[QT][SUB];
        tile.template scores<QT>([&](int y, int c) { return qf[y][c]; }, sc, gq, row_bytes);
        if (tt == 0) next();  // (under the products)
        const uint32_t gone = (uint32_t)(gone_s >> (tt * TILE)) & (uint32_t)((1ull << TILE) - 1);
        const uint32_t va[4] = {base + v_at[0], base + v_at[1], base + v_at[2], base + v_at[3]};
        const auto read_v = [&](auto ng) {
          uint32_t* const o[8] = {tile.v[0][0][ng], tile.v[0][1][ng], tile.v[0][2][ng], tile.v[0][3][ng],
                                  tile.v[SUB - 1][0][ng], tile.v[SUB - 1][1][ng], tile.v[SUB - 1][2][ng], tile.v[SUB - 1][3][ng]};
          lds_read<G::VB / 4, 16 * G::VB * ng, SUB == 2 ? 16 * G::VB * ng + 16 * S::ROW : 0>(va, o);
        };
        read_v(std::integral_constant<int, 0>{});
        if constexpr (G::NG > 1) read_v(std::integral_constant<int, 1>{});
        if constexpr (G::NG > 2) read_v(std::integral_constant<int, 2>{}), read_v(std::integral_constant<int, 3>{});
        // positions that not all columns see
        const bool cut = t + TILE > n_min || gone;
        bool odd = false;  // some of what only some columns see is not finite
        if (cut) {
#pragma unroll
          for (int sb = 0; sb < SUB; ++sb)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int p = 16 * sb + 4 * gq + j;
              const bool off = gone >> p & 1;
#pragma unroll
              for (int y = 0; y < QT; ++y)
                if (t + p >= my_n[y] || off) sc[y][sb][j] = -INFINITY;
              if (t + p >= n_max || off) tile.clear_v(sb, j);
              if (t + p >= n_min) {
#pragma unroll
                for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
                  for (int e = 0; e < G::VB / 4; ++e) {
                    odd |= sh_finite<G::ES>(tile.v[sb][j][ng][e]);
                  }
              }
            }
          odd = __any(odd);
        }
#pragma unroll
        for (int y = 0; y < QT; ++y) sh_weights<G>(A, sc[y], mx[y], l[y], acc[y]);
        tile.template weigh<QT, false, true>(sc, acc);
        const char* vp = s_kv[s % S::RING] + S::BYTES + tt * TILE * S::ROW;
        if (odd) {  // what was left out, for those who see it: the sum is not finite there, whatever the weight
#pragma unroll 1
          for (int p = max(0, n_min - t); p < min(TILE, n_max - t); ++p) {
            if (gone >> p & 1) continue;
#pragma unroll
            for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int b16 = (16 * ng + 4 * gq + r) * G::VB;  // (bytes of the row)
                const char* v = vp + p * S::ROW + 16 * sh_slot<S::ROW>(p, b16 / 16) + b16 % 16;
#pragma unroll
                for (int y = 0; y < QT; ++y) sh_add_odd<G>(v, t + p < my_n[y], acc[y][ng], r);
              }
          }
        }
      }
    }

    // ---- the piece's sums to its slot ----
    float* out = A.seeds + (((int64_t)(gang + x) * A.gang + member) * pw + wp) * COLS * (DP + 4);
#pragma unroll
    for (int y = 0; y < QT; ++y) {
      float sum = l[y];
      sum += __shfl_xor(sum, 16, 64);
      sum += __shfl_xor(sum, 32, 64);
      const int c = (wc * QT + y) * 16 + m16;
      float* o = out + (int64_t)c * (DP + 4);
      const bool sees = my_n[y] > 0;  // (others: sums of nothing)
      if (ct * COLS + c >= q.rows * A.heads) continue;
#pragma unroll
      for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int e = 0; e < G::VD; e += 4)
            stg4(o + 16 * G::VD * ng + G::VD * (4 * gq + r) + e,
                 sees ? f32x4{acc[y][ng][e][r], acc[y][ng][e + 1][r], acc[y][ng][e + 2][r], acc[y][ng][e + 3][r]}
                      : f32x4{0.f, 0.f, 0.f, 0.f});
      if (gq == 0) stg4(o + DP, f32x4{sees ? mx[y] : -INFINITY, sees ? sum : 0.f, 0.f, 0.f});
    }
  }
}

// Sums over what the rows of a run hold of their own, for a chunk of their tiles: a
// wave a piece, as K and V stream by; few columns, so bound by the memory.
template <typename T, int DP, bool PAGE16, bool EXACT>
__device__ __forceinline__ void sh_own(const SharedArgs& A, const ShCall& call, const ShShared& L, uint32_t chunk, uint32_t each) {
  using G = AttGeo<T, DP>;
  using S = ShGeo<T, DP>;
  constexpr int TILE = G::TILE, SUB = G::SUB;
  const int lane = threadIdx.x & 63, m16 = lane & 15, gq = lane >> 4;
  const int D = EXACT ? DP : A.head_dim, row_bytes = D * G::ES, H = A.n_kv * A.q_tiles;
  const uint32_t total = L.t[256] * H;
  const uint32_t u_end = (uint32_t)min((uint64_t)total, (uint64_t)(chunk + 1) * each);
  const uint32_t neg = A.negate ? (G::ES == 2 ? 0x80008000u : 0x80000000u) : 0u;
  const uint32_t tok = (uint32_t)A.token_stride * G::ES;
  const auto page_of = [&](int t) { return (int)(((uint64_t)(uint32_t)t * A.ps_mul) >> (31 + A.ps_shift)); };
  for (uint32_t u = (uint32_t)min((uint64_t)total, (uint64_t)chunk * each); u < u_end;) {
    // the run that holds unit u
    const int lo = sh_find(L.t, u / in_place(H));
    uint32_t before = L.t[lo];
    ShRun R{};
    for (int base = lo * call.per_r; base < A.n_rows && R.tiles == 0; base += A.together)  // (the next border is past u)
      sh_runs<S, TILE>(A, call, L, base, [&](const ShRun& r) {
        if (R.tiles == 0) {
          if (u < (before + r.tiles) * H)
            R = r;
          else
            before += r.tiles;
        }
      });
    R = {uni(R.row), uni(R.rows), uni(R.req), uni(R.lo), uni(R.n), uni(R.every_lo), uni(R.every_n), uni(R.tiles)};
    before = (uint32_t)uni((int)before);
    if (R.tiles == 0) return;  // (only if the lengths change while the call runs)
    const uint32_t in = u - before * H;
    const int hh = in / in_place(R.tiles), ta = in - hh * R.tiles, cnt = min((uint32_t)(R.tiles - ta), u_end - u);
    const int kvh = A.q_tiles == 1 ? hh : hh / in_place(A.q_tiles), qt = hh - kvh * A.q_tiles;
    u += cnt;
    // columns: c is head h0 + c % wide of row c / wide
    const bool several = A.together > 1;
    const int wide = several ? A.heads : 16, nq = several ? R.rows * A.heads : min(16, A.heads - 16 * qt);
    const int h0 = kvh * A.heads + 16 * qt, col = min(m16, nq - 1), my_row = several ? col / in_place(wide) : 0;
    int my_n = R.n, my_lo = R.lo;
    if (R.rows > 1) {
      my_n = sh_len(A, R.row + my_row);
      my_lo = min(my_n, sh_from<S>(A, call, L, R.row + my_row));
    }
    const char* qp = (const char*)A.q + ((int64_t)(R.row + my_row) * A.q_stride + (int64_t)(h0 + col - my_row * wide) * D) * G::ES;
    uint4 q[G::NC];
#pragma unroll
    for (int c = 0; c < G::NC; ++c) {
      const int at = 64 * c + 16 * gq;
      const uint4 x = ldg_b16<false>(qp, EXACT ? at : min(at, row_bytes - 16));
      q[c] = m16 < nq && (EXACT || at < row_bytes) ? make_uint4(x.x ^ neg, x.y ^ neg, x.z ^ neg, x.w ^ neg) : make_uint4(0, 0, 0, 0);
    }
    const char *kb = (const char*)A.k, *vb = (const char*)A.v;
    const int32_t* tab = A.table + (int64_t)R.req * A.table_stride;
    const int64_t head = (int64_t)kvh * A.head_stride * G::ES;
    const int tb = R.lo / TILE + ta;

    AttTile<T, DP, EXACT> tile;
    int32_t place_lo[SUB], place_hi[SUB], page_next[SUB];
    const auto look_up = [&](int i) {
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        if constexpr (PAGE16) {  // the next 64 tiles' blocks, a tile a lane
          const int t = min((tb + i + lane) * TILE + 16 * s, (R.n - 1) & ~15);
          const int at = page_of(t), page = ldg(tab + at);
          const int64_t off = ((int64_t)page * A.page_stride + (int64_t)(t - at * A.page_size) * A.token_stride) * G::ES + head;
          const bool ok = page >= 0 && page < A.n_pages;
          place_lo[s] = ok ? (int32_t)(uint32_t)off : -1;
          place_hi[s] = ok ? (int32_t)(off >> 32) : -1;
        } else {  // the tile's positions, one a lane
          page_next[s] = ldg(tab + page_of(min((tb + i) * TILE + 16 * s + m16, R.n - 1)));
        }
      }
    };
    int64_t off[SUB];
    uint32_t bad[SUB];
    const auto locate = [&](int i) {
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        if constexpr (PAGE16) {
          const int src = i & 63;
          const int64_t o = (int64_t)(((uint64_t)(uint32_t)lane_of(place_hi[s], src) << 32) | (uint32_t)lane_of(place_lo[s], src));
          bad[s] = o < 0 ? 0xFFFFu : 0u;
          off[s] = o < 0 ? head : o;
        } else {
          const int t = min((tb + i) * TILE + 16 * s + m16, R.n - 1), page = page_next[s];
          const bool ok = page >= 0 && page < A.n_pages;
          off[s] = (ok ? ((int64_t)page * A.page_stride + (int64_t)(t - page_of(t) * A.page_size) * A.token_stride) * G::ES : 0) + head;
          bad[s] = (uint32_t)(__ballot(!ok) & 0xFFFFu);
        }
      }
    };
    const auto load_k = [&]() {
#pragma unroll
      for (int s = 0; s < SUB; ++s)
#pragma unroll
        for (int c = 0; c < G::NC; ++c) {
          if (!EXACT && DP > 64 && 64 * c >= row_bytes) continue;  // (uniform)
          const uint32_t at = EXACT ? 64 * c + 16 * gq : min(64 * c + 16 * gq, row_bytes - 16);
          tile.k[s][c] = ldg_b16<true>(kb + off[s], PAGE16 ? m16 * tok + at : at);
        }
    };
    const auto load_v = [&]() {
#pragma unroll
      for (int s = 0; s < SUB; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const char* p = vb + off[s];
          uint32_t o = (4 * gq + j) * tok;
          if constexpr (!PAGE16) {
            const int src = 4 * gq + j;
            const uint32_t lo32 = __shfl((int)(uint32_t)off[s], src, 64), hi32 = __shfl((int)(off[s] >> 32), src, 64);
            p = vb + (int64_t)(((uint64_t)hi32 << 32) | lo32);
            o = 0;
          }
#pragma unroll
          for (int ng = 0; ng < G::NG; ++ng) {
            const int at = (16 * ng + m16) * G::VB;
            tile.template load_v<true>(p, o + (EXACT ? at : min(at, row_bytes - G::VB)), s, j, ng);
          }
        }
    };

    float mx[1] = {-INFINITY}, l = 0.f;
    f32x4 acc[1][G::NG][G::VD];
#pragma unroll
    for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
      for (int e = 0; e < G::VD; ++e) acc[0][ng][e] = f32x4{0.f, 0.f, 0.f, 0.f};
    look_up(0);
    locate(0);
    load_k();
    load_v();
    if constexpr (!PAGE16) look_up(min(1, cnt - 1));
    // (the next tile's loads run under this one's products)
    const auto trip = [&](int i, auto more) {
      const int t = (tb + i) * TILE;
      uint32_t gone[SUB];
      bool cut = t < R.every_lo || t + TILE > R.every_n;
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        gone[s] = bad[s];
        cut = cut || bad[s] != 0;
      }
      f32x4 sc[1][SUB];
      tile.template scores<1>([&](int, int c) { return q[c]; }, sc, gq, row_bytes);
      if constexpr (more) {
        if constexpr (PAGE16) {
          if (((i + 1) & 63) == 0) look_up(i + 1);
        }
        locate(i + 1);
        load_k();
        if constexpr (!PAGE16) look_up(min(i + 2, cnt - 1));
      }
      bool odd = false;
      if (cut) {
        // a position that is not seen has no weight; what is not finite where only
        // some rows see it is left out and added for those below
#pragma unroll
        for (int s = 0; s < SUB; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = t + 16 * s + 4 * gq + j;
            const bool away = gone[s] >> (4 * gq + j) & 1;
            if (at < my_lo || at >= my_n || away) sc[0][s][j] = -INFINITY;
            if (at < R.lo || at >= R.n || away) tile.clear_v(s, j);
            if (at < R.every_lo || at >= R.every_n) {
#pragma unroll
              for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
                for (int e = 0; e < G::VB / 4; ++e) odd |= sh_finite<G::ES>(tile.v[s][j][ng][e]);
            }
          }
        odd = __any(odd);
      }
      sh_weights<G>(A, sc[0], mx[0], l, acc[0]);
      tile.template weigh<1, false, true>(sc, acc);
      if (odd) {
        for (int p = 0; p < TILE; ++p) {
          const int at = t + p, sub = SUB == 2 ? p >> 4 : 0;
          if ((at >= R.every_lo && at < R.every_n) || at < R.lo || at >= R.n || (gone[sub] >> (p & 15) & 1)) continue;
          const int c = page_of(at), page = ldg(tab + c);
          const char* row = vb + ((int64_t)page * A.page_stride + (int64_t)(at - c * A.page_size) * A.token_stride) * G::ES + head;
#pragma unroll
          for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int b = (16 * ng + 4 * gq + r) * G::VB;
              sh_add_odd<G>(row + (EXACT ? b : min(b, row_bytes - G::VB)), at >= my_lo && at < my_n, acc[0][ng], r);
            }
        }
      }
      if constexpr (more) load_v();
    };
    for (int i = 0; i + 1 < cnt; ++i) trip(i, std::true_type());
    trip(cnt - 1, std::false_type());

    // ---- the piece's sums to its slot ----
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    float* o = A.own + ((int64_t)chunk + (int64_t)R.row * H + hh) * A.own_cols * (DP + 4) + m16 * (DP + 4);
    if (m16 < nq) {
      const bool sees = my_n > my_lo;  // (others: sums of nothing)
#pragma unroll
      for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int e = 0; e < G::VD; e += 4)
            stg4(o + 16 * G::VD * ng + G::VD * (4 * gq + r) + e,
                 sees ? f32x4{acc[0][ng][e][r], acc[0][ng][e + 1][r], acc[0][ng][e + 2][r], acc[0][ng][e + 3][r]}
                      : f32x4{0.f, 0.f, 0.f, 0.f});
      if (gq == 0) stg4(o + DP, f32x4{sees ? mx[0] : -INFINITY, sees ? l : 0.f, 0.f, 0.f});
    }
  }
}

// Both kinds of work at once: products over shared positions keep the matrix
// units busy while what the rows have of their own streams from memory.
//
// How the work is cut. A unit is one stage of positions of one (group, key head,
// wide tile of columns): as many tiles of 128 columns as a gang has work-groups,
// which lie on one die and walk the positions side by side, so that all but the
// first find them in its L2. The units, numbered in that order, are cut into
// equal ranges for the gangs; so are the tiles of positions of all (row, head)s
// for the waves of the other work-groups. Gang or wave w's part of the x-th
// (group, key head, wide tile) or (row, head) is a piece, in slot w + x: both grow
// from piece to piece, so slots are not shared and those of one x lie side by
// side. Lengths and groups are on the device; every work-group numbers them by
// itself, and the partial results are joined by the next launch.
//
// 8 x 64 rows behind 32000 shared positions, 32 heads of 128 over 8, bf16: 947 us and
// 17 of the join, 415 GF and 2.4 GB (438 TFLOP/s of products, 30% of the matrix
// units' cycles); 128 rows of one group behind 8192: 76 and 7. What bounds it: the
// softmax of a score costs as many cycles as its products, and both wait for LDS;
// the prefix alone takes 740 us, without the softmax 630, without V's products 536.
template <typename T, int DP, bool PAGE16, bool EXACT>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void k_shared_attention(SharedArgs A) {
  using G = AttGeo<T, DP>;
  using S = ShGeo<T, DP>;
  __shared__ __align__(1024) char s_kv[S::RING][2 * S::BYTES];
  __shared__ ShShared L;
  const int tid = threadIdx.x, lane = tid & 63, w = uni(tid >> 6);
  ShCall call;
  call.per_g = (A.n_groups + 255) / 256;
  call.per_r = ((A.n_rows + 255) / 256 + A.together - 1) / A.together * A.together;
  // ---- the groups ----
  {
    uint32_t u = 0, x = 0;
    // (the first 256 threads' groups, and rows below)
    if (tid < 256) L.row[tid] = A.n_rows, L.end[tid] = 0, L.n[tid] = 0;
    const int g0 = min(A.n_groups, tid * call.per_g), g1 = min(A.n_groups, g0 + call.per_g);
    for (int g = g0; g < g1; ++g) {
      const ShGroup q = sh_group<S>(A, g);
      if (g == g0) L.row[tid] = q.row, L.end[tid] = q.row + q.rows, L.n[tid] = q.n;
      u += (uint32_t)q.units * q.tiles * A.n_kv;
      x = (uint32_t)min((int64_t)SH_TILES, x + (int64_t)(q.units ? q.tiles : 0) * A.n_kv);
    }
    const uint32_t iu = wave_scan(u), ix = wave_scan(x);
    if (lane == 63 && w < 4) L.sum[0][w] = iu, L.sum[1][w] = ix;
    __syncthreads();
    uint32_t bu = 0, bx = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < w) bu += L.sum[0][i], bx += L.sum[1][i];
    if (tid < 256) L.u[tid + 1] = bu + iu, L.x[tid + 1] = bx + ix;
    if (tid == 0) L.u[0] = L.x[0] = 0;
    __syncthreads();
  }
  // groups that overlap may be more tiles than the workspace has room for: then
  // nothing is shared (below that the units are under 2^31)
  call.fits = L.x[256] <= (uint32_t)A.max_tiles;
  // ---- the rows ----
  {
    uint32_t t = 0;
    const int r0 = min(A.n_rows, tid * call.per_r), r1 = min(A.n_rows, r0 + call.per_r);
    for (int r = r0; r < r1; r += A.together) sh_runs<S, G::TILE>(A, call, L, r, [&](const ShRun& q) { t += q.tiles; });
    const uint32_t it = wave_scan(t);
    if (lane == 63 && w < 4) L.sum[0][w] = it;
    __syncthreads();
    uint32_t bt = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < w) bt += L.sum[0][i];
    if (tid < 256) L.t[tid + 1] = bt + it;
    if (tid == 0) L.t[0] = 0;
    __syncthreads();
  }
  const int H = A.n_kv * A.q_tiles;
  const uint32_t units = call.fits ? L.u[256] : 0, tiles = L.t[256] * H;
  // ---- shares of the work-groups ----
  const ShCut cut = sh_cut(gridDim.x, units, tiles, A.gang, A.pw);
  // (whole gangs on each of the dies, to which work-groups go in turn)
  const uint32_t die = blockIdx.x % cut.dies, k = blockIdx.x / cut.dies;
  // ---- where each row's partial results will lie ----
  if (blockIdx.x == 0 && tid == 0) A.plan->each_shared = cut.each_s, A.plan->each_own = cut.each_o;
  for (int base = (blockIdx.x * 64 * S::NW + tid) * A.together; base < A.n_rows; base += gridDim.x * 64 * S::NW * A.together) {
    const int chunk = base / call.per_r;
    uint32_t before = L.t[chunk];
    for (int b = chunk * call.per_r; b < base; b += A.together)
      sh_runs<S, G::TILE>(A, call, L, b, [&](const ShRun& q) { before += q.tiles; });
    sh_runs<S, G::TILE>(A, call, L, base, [&](const ShRun& q) {
      for (int i = 0; i < q.rows; ++i) {
        ShRow R{0, 0, 0, 0, 0, q.tiles, before, q.row, A.together > 1 ? i * A.heads : 0, {0, 0, 0}};
        sh_group_of<S>(A, call, L, q.row + i, [&](const ShGroup& g, uint32_t u, uint32_t x) {
          R.units = g.units, R.tiles = g.tiles, R.col0 = (q.row + i - g.row) * A.heads, R.u0 = u, R.x0 = x;
        });
        A.rows[q.row + i] = R;
      }
      before += q.tiles;
    });
  }
  // ---- the work-groups' kinds, spread evenly ----
  const uint32_t upto = k * cut.ws / cut.here, next = (k + 1) * cut.ws / cut.here;
  if (next > upto) {
    sh_prefix<T, DP, PAGE16, EXACT>(A, call, L, s_kv, die * (cut.ws / A.gang) + upto / A.gang, (int)(upto % A.gang), cut.each_s);
  } else {
    for (uint32_t chunk = S::NW * (die * cut.wo + k - upto) + w; chunk < cut.chunks;) {
      sh_own<T, DP, PAGE16, EXACT>(A, call, L, chunk, cut.each_o);
      int taken = 0;
      if (lane == 0) taken = arrive(&A.plan->taken);
      chunk = cut.waves + (uint32_t)uni(taken);
    }
  }
}

// The slots of a (row, head), DP / 4 lanes for its elements, eight slots' loads in
// flight: shared positions' first, each in the work's order, so the result does
// not depend on who was done when.
template <typename T, int DP>
__global__ __launch_bounds__(256) void k_shared_join(SharedArgs A) {
  using S = ShGeo<T, DP>;
  constexpr int LP = DP / 4;
  const int n_heads = A.n_kv * A.heads, H = A.n_kv * A.q_tiles, d = 4 * (threadIdx.x % LP);
  const ShPlan P = *A.plan;
  if (blockIdx.x == 0 && threadIdx.x == 0) A.plan->taken = 0;
  if (d >= A.head_dim) return;
  for (int64_t pair = (int64_t)blockIdx.x * (256 / LP) + threadIdx.x / LP; pair < (int64_t)A.n_rows * n_heads;
       pair += (int64_t)gridDim.x * (256 / LP)) {
    const int row = (int)(pair / n_heads), h = (int)(pair - (int64_t)row * n_heads);
    const ShRow R = A.rows[row];
    const int kvh = h / A.heads, hg = h - kvh * A.heads;
    // shared
    const int COLS = S::WCOLS * A.cw, c = R.col0 + hg, ct = c / COLS;
    const uint32_t x = (uint32_t)(kvh * R.tiles + ct / A.gang), u = R.u0 + x * R.units, w0 = u / P.each_shared;
    const int n0 = R.units ? ((int)((u + R.units - 1) / P.each_shared - w0) + 1) * A.pw : 0;
    const float* p0 = A.seeds + (((int64_t)(w0 + R.x0 + x) * A.gang + ct % A.gang) * A.pw * COLS + c % COLS) * (DP + 4);
    // own
    const int qt = A.together > 1 ? 0 : hg / 16, hh = kvh * A.q_tiles + qt, col = R.at + hg - 16 * qt;
    const uint32_t v = R.before * H + (uint32_t)hh * R.own, w1 = v / P.each_own;
    const int n1 = R.own ? (int)((v + R.own - 1) / P.each_own - w1) + 1 : 0;
    const float* p1 = A.own + ((int64_t)w1 + (int64_t)R.lead * H + hh) * A.own_cols * (DP + 4) + col * (DP + 4);
    // (slots of one x: its turns lie side by side, its pieces a gang's slots apart)
    const int64_t turn = (int64_t)COLS * (DP + 4), s0 = A.gang * A.pw * turn, s1 = (int64_t)A.own_cols * (DP + 4);
    float m = -INFINITY, l = 0.f;
    f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < n0 + n1; j0 += 8) {
      f32x4 ml[8], z[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = min(j0 + j, n0 + n1 - 1);
        const float* p = i < n0 ? p0 + i / A.pw * s0 + i % A.pw * turn : p1 + (i - n0) * s1;
        ml[j] = ldg4(p + DP);
        z[j] = ldg4(p + d);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j0 + j >= n0 + n1) break;
        const float mn = fmaxf(m, ml[j].x), ref = mn == -INFINITY ? 0.f : mn;
        const float fa = __builtin_amdgcn_exp2f(m - ref), fb = __builtin_amdgcn_exp2f(ml[j].x - ref);
        o = o * fa + z[j] * fb;
        l = l * fa + ml[j].y * fb;
        m = mn;
      }
    }
    const f32x4 y = l == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : o / l;
    const int64_t at = (int64_t)row * A.out_stride + (int64_t)h * A.head_dim + d;
    if constexpr (sizeof(T) == 4) {
      stg4((float*)A.out + at, y);
    } else {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      *(GLOBAL u32x2*)((uint16_t*)A.out + at) = u32x2{pack_bf2(__float_as_uint(y.x), __float_as_uint(y.y)),
                                                     pack_bf2(__float_as_uint(y.z), __float_as_uint(y.w))};
    }
  }
}

template <typename T, int DP>
void sh_launch(const SharedArgs& A, int blocks, hipStream_t s) {
  const dim3 threads(256);
  if (A.page_size % 16)
    hipLaunchKernelGGL((k_shared_attention<T, DP, false, false>), dim3(blocks), threads, 0, s, A);
  else if (A.head_dim == DP)
    hipLaunchKernelGGL((k_shared_attention<T, DP, true, true>), dim3(blocks), threads, 0, s, A);
  else
    hipLaunchKernelGGL((k_shared_attention<T, DP, true, false>), dim3(blocks), threads, 0, s, A);
  const int64_t pairs = (int64_t)A.n_rows * A.n_kv * A.heads;
  hipLaunchKernelGGL((k_shared_join<T, DP>), dim3((unsigned)sh_join_blocks(pairs, DP)), dim3(256), 0, s, A);
}
template <typename T>
void sh_dim(const SharedArgs& A, int dp, int blocks, hipStream_t s) {
  if (dp == 64) sh_launch<T, 64>(A, blocks, s);
  else if (dp == 128) sh_launch<T, 128>(A, blocks, s);
  else sh_launch<T, 256>(A, blocks, s);
}

}  // namespace scute

using namespace scute;

extern "C" scute_status scute_shared_attention_workspace(int32_t device, int32_t dtype, int32_t head_dim,
                                                         int32_t n_heads, int32_t n_kv_heads, int32_t max_rows,
                                                         int32_t max_groups, int64_t* bytes) {
  const char* fn = "scute_shared_attention_workspace";
  const auto bad = [&](scute_status code, const char* what) { return fail(code, std::string(fn) + ": " + what); };
  if (!bytes) return bad(SCUTE_E_INVALID, "bytes is null");
  if (device < 0) return bad(SCUTE_E_INVALID, "device must be >= 0");
  if (dtype != SCUTE_BF16 && dtype != SCUTE_F32) return bad(SCUTE_E_INVALID, "dtype must be SCUTE_BF16 or SCUTE_F32");
  if (head_dim < 8 || head_dim > 256 || head_dim % 8) return bad(SCUTE_E_SHAPE, "head_dim must be a multiple of 8 in [8, 256]");
  if (n_kv_heads < 1 || n_kv_heads > 1024 || n_heads < 1 || n_heads > 65536 || n_heads % n_kv_heads)
    return bad(SCUTE_E_SHAPE, "n_heads must be a multiple of n_kv_heads in [1, 65536], n_kv_heads in [1, 1024]");
  if (max_rows < 0 || max_rows > (1 << 20) || max_groups < 0 || max_groups > 65536)
    return bad(SCUTE_E_SHAPE, "max_rows must be in [0, 2^20] and max_groups in [0, 65536]");
  const int units = device_units(device);
  if (units < 0) return bad(SCUTE_E_INVALID, "no such HIP device");
  *bytes = sh_workspace(dtype == SCUTE_F32 ? 4 : 2, att_dim(head_dim), att_workspace(units, head_dim), sizeof(ShRow), n_heads,
                        n_kv_heads, max_rows, max_groups, units);
  return SCUTE_OK;
}

extern "C" scute_status scute_shared_attention(const scute_kv_cache* C, const void* q, int64_t q_stride,
                                               int32_t n_heads, const int32_t* table, int64_t table_stride,
                                               int32_t n_requests, int32_t table_width, const int32_t* len,
                                               const int32_t* req, int32_t n_rows, const int32_t* group,
                                               const int32_t* shared_len, int32_t n_groups, float scale, void* out,
                                               int64_t out_stride, void* workspace, int64_t workspace_bytes,
                                               uint32_t flags, void* stream) {
  const char* fn = "scute_shared_attention";
  const auto bad = [&](scute_status code, const char* what) { return fail(code, std::string(fn) + ": " + what); };
  const AttCall call{C, q, q_stride, n_heads, table, table_stride, n_requests, table_width, len, req, n_rows, scale,
                     0, 0, out, out_stride, workspace, workspace_bytes};
  const scute_status st = att_check(fn, call);
  if (st != SCUTE_OK) return st;
  if (flags & ~(uint32_t)SCUTE_SHARED_ALWAYS) return bad(SCUTE_E_INVALID, "unknown flag");
  if (n_groups < 0 || n_groups > 65536) return bad(SCUTE_E_SHAPE, "n_groups must be in [0, 65536]");
  if (n_rows == 0) return SCUTE_OK;
  if (n_groups > 0 && (!group || !shared_len)) return bad(SCUTE_E_INVALID, "null pointer");
  if (((uintptr_t)group | (uintptr_t)shared_len) & 3) return bad(SCUTE_E_INVALID, "misaligned pointer");
  OnDevice g(C->device);
  if (!g.ok()) return hip_fail(g.err, fn);
  const int units = device_units(C->device);
  if (units < 0) return bad(SCUTE_E_INVALID, "no such HIP device");
  const int es = C->dtype == SCUTE_F32 ? 4 : 2, dp = att_dim(C->head_dim);
  // (paged attention's workspace comes first, for calls that share nothing; its
  // counters hold the plan, which has to stay as the last call left it)
  const ShSizes z = sh_sizes(es, dp, att_workspace(units, C->head_dim), sizeof(ShRow), C->page_size, n_heads, C->n_kv_heads,
                             req != nullptr, n_rows, n_groups, units);
  if (workspace_bytes < z.bytes) return bad(SCUTE_E_INVALID, "the workspace is too small");
  const int64_t reach = std::min<int64_t>((int64_t)table_width * C->page_size, (int64_t)1 << 29);
  // Sharing has more to do before and after than paged attention of few rows, whose
  // reads it saves. Where it cannot save as much, at the table's whole width, the rows
  // are read for one by one (captured calls, shared and one by one: 4 rows behind 8000
  // positions, 97 MB, 51 and 29 us; 32 behind 1000, 130 MB, 44 and 21; 4 behind 32000,
  // 390 MB, 74 and 80).
  const int64_t saved = std::max<int64_t>(0, (int64_t)n_rows - n_groups) * reach * 2 * C->n_kv_heads * C->head_dim * es;
  if ((!(flags & SCUTE_SHARED_ALWAYS) && (n_groups == 0 || saved < SH_SAVED)) || !sh_can_share(z))
    return att_run(fn, call, ATT_PLAIN, (hipStream_t)stream);
  // (units and tiles are counted in 31 bits)
  const int64_t stage = es == 4 ? 16 : 32, most = ((int64_t)1 << 31) - 1;
  if (z.tiles >= SH_TILES || z.tiles * (reach / stage + 1) > most ||
      (int64_t)n_rows * C->n_kv_heads * z.q_tiles * (reach / stage + 2) > most)
    return bad(SCUTE_E_SHAPE, "too many rows and heads for a table this wide");
  char* ws = (char*)workspace;
  int shift = 0;
  while ((1 << shift) < C->page_size) ++shift;
  const uint64_t mul = (((uint64_t)1 << (31 + shift)) + C->page_size - 1) / C->page_size;
  const SharedArgs A{q, C->k, C->v, out, table, len, req, group, shared_len, (ShRow*)(ws + z.rows), (ShPlan*)(ws + att_plan_place(units)),
                     (float*)(ws + z.seeds), (float*)(ws + z.own), q_stride, out_stride, C->page_stride, C->token_stride,
                     C->head_stride, table_stride, C->n_pages, (uint32_t)mul, n_rows, n_groups, C->n_kv_heads, z.group,
                     C->head_dim, C->page_size, shift, (int32_t)reach, n_requests, (int32_t)z.tiles, z.cw, z.pw, z.gang, z.together, z.q_tiles,
                     z.own_cols, scale < 0.f, std::max(fabsf(scale * 1.4426950408889634f), 1e-37f)};
  const hipStream_t s = (hipStream_t)stream;
  if (es == 4) sh_dim<float>(A, dp, z.blocks, s);
  else sh_dim<uint16_t>(A, dp, z.blocks, s);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SCUTE_OK : hip_fail(e, fn);
}
