// Attention of rows whose contexts begin with the same positions
// (scute_shared_attention): the shared positions once for all rows of a group,
// here; what each row has beside them by the kernel of attend.h, which joins
// the two.

#include <algorithm>

#include "attend.h"
#include "attend_host.h"

namespace scute {

struct SharedArgs {
  const void *q, *k, *v;
  const int32_t *table, *len, *req, *group, *shared;
  AttRowFrom* from;
  float* seeds;
  int64_t q_stride, page_stride, token_stride, head_stride, table_stride, n_pages;
  uint32_t ps_mul;
  int32_t n_rows, n_groups, n_kv, heads, head_dim, page_size, ps_shift, reach, n_requests, max_tiles;
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
  static constexpr int COLS = 4 * 16 * QT;               // columns of a work-group
  static constexpr int ROW = DP * G::ES;                 // bytes of a position in LDS
  static constexpr int STAGE = sh_stage(G::ES, DP);      // positions staged at once: a unit
  static constexpr int RING = 4, BYTES = STAGE * ROW;    // stages of K (and of V) in LDS
  static constexpr int PIECES = ROW / 16;                // 16-byte pieces of a position
  static constexpr int LOADS = BYTES / 4096;             // a wave's loads of 1 KB a stage (of K, and of V)
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

constexpr int SH_TILES = 1 << 22;  // (group, key head, tile)s stay below it

struct ShGroup {
  int row, rows, n, tiles, units;  // first row, rows, shared positions, column tiles, units of positions
};
template <typename S>
__device__ __forceinline__ ShGroup sh_group(const SharedArgs& A, int g) {
  ShGroup q;
  const int a = min(max(ldg(A.group + g), 0), A.n_rows), b = min(max(ldg(A.group + g + 1), 0), A.n_rows);
  q.row = a, q.rows = max(b - a, 0);
  q.n = min(max(ldg(A.shared + g), 0), A.reach);
  q.tiles = (int)(((int64_t)q.rows * A.heads + S::COLS - 1) / S::COLS);
  q.units = (q.n + S::STAGE - 1) / S::STAGE;
  return q;
}
__device__ __forceinline__ int sh_len(const SharedArgs& A, int row) {
  const int len = ldg(A.len + row), req = A.req ? ldg(A.req + row) : row;
  return (uint32_t)req < (uint32_t)A.n_requests ? min(max(len, 0), A.reach) : 0;
}

// Sums of the softmax over a group's shared positions for all its rows: a
// product of tall matrices, so K and V go through LDS once for 128 columns (rows
// times the heads of a key head), 32 columns a wave, and a wave's columns are
// its own: nothing is joined between waves.
//
// How the work is cut. A unit is one stage of positions of one (group, key head,
// tile of columns); the units are numbered in that order and every work-group
// takes the same number of consecutive ones. Work-group w's part of the x-th
// (group, key head, tile) is a piece, in slot w + x: both grow from piece to
// piece, so slots are not shared and a (group, key head, tile)'s lie side by
// side. Lengths and groups are on the device; every work-group numbers them by
// itself.
template <typename T, int DP, bool EXACT>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void k_shared_prefix(SharedArgs A) {
  using G = AttGeo<T, DP>;
  using S = ShGeo<T, DP>;
  constexpr int TILE = G::TILE, SUB = G::SUB, QT = S::QT, COLS = S::COLS;
  __shared__ __align__(1024) char s_kv[S::RING][2 * S::BYTES];
  __shared__ uint32_t s_u[257], s_x[257];   // units and (group, key head, tile)s before each thread's groups
  __shared__ int s_row[257];                // their first row
  __shared__ uint32_t s_sum[2][4];
  __shared__ unsigned long long s_lead[4];
  const int tid = threadIdx.x, lane = tid & 63, w = uni(tid >> 6), m16 = lane & 15, gq = lane >> 4;
  const int D = EXACT ? DP : A.head_dim, row_bytes = D * G::ES;

  // ---- the numbering ----
  const int per = (A.n_groups + 255) / 256, g0 = min(A.n_groups, tid * per), g1 = min(A.n_groups, g0 + per);
  {
    uint32_t u = 0, x = 0;
    for (int g = g0; g < g1; ++g) {
      const ShGroup q = sh_group<S>(A, g);
      if (g == g0) s_row[tid] = q.row;
      u += (uint32_t)q.units * q.tiles * A.n_kv;
      x = (uint32_t)min((int64_t)SH_TILES, x + (int64_t)(q.units ? q.tiles : 0) * A.n_kv);
    }
    if (g0 >= g1) s_row[tid] = A.n_rows;
    const uint32_t iu = wave_scan(u), ix = wave_scan(x);
    if (lane == 63) s_sum[0][w] = iu, s_sum[1][w] = ix;
    __syncthreads();
    uint32_t bu = 0, bx = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < w) bu += s_sum[0][i], bx += s_sum[1][i];
    s_u[tid + 1] = bu + iu, s_x[tid + 1] = bx + ix;
    if (tid == 0) s_u[0] = s_x[0] = 0;
    __syncthreads();
  }
  // groups that overlap may be more tiles than the workspace has room for: then
  // nothing is shared (below that the units are under 2^31)
  const bool fits = s_x[256] <= (uint32_t)A.max_tiles;
  const uint32_t total = fits ? s_u[256] : 0, each = total ? (total + gridDim.x - 1) / gridDim.x : 1;

  // ---- where each row's partial results will lie ----
  for (int row = blockIdx.x * 256 + tid; row < A.n_rows; row += gridDim.x * 256) {
    int lo = 0;  // the last thread whose groups begin at or before the row
    for (int step = 128; step > 0; step >>= 1)
      if (s_row[lo + step] <= row) lo += step;
    uint32_t u = s_u[lo], x = s_x[lo];
    AttRowFrom F{0, 0, 0, 0, 0, 0, 0, 0};
    for (int g = lo * per; fits && g < min(A.n_groups, lo * per + per); ++g) {
      const ShGroup q = sh_group<S>(A, g);
      if (row >= q.row && row < q.row + q.rows) {
        F.from = q.n, F.tiles = q.tiles, F.col0 = (row - q.row) * A.heads;
        F.u0 = u, F.x0 = x, F.units = q.units, F.each = each;
        break;
      }
      u += (uint32_t)q.units * q.tiles * A.n_kv;
      x += (uint32_t)(q.units ? q.tiles : 0) * A.n_kv;
    }
    A.from[row] = F;
  }

  // ---- this work-group's units ----
  const uint32_t u_end = min((uint64_t)total, (uint64_t)(blockIdx.x + 1) * each);
  for (uint32_t u = min((uint64_t)total, (uint64_t)blockIdx.x * each); u < u_end;) {
    int lo = 0;
    for (int step = 128; step > 0; step >>= 1)
      if (s_u[lo + step] <= u) lo += step;
    uint32_t u0 = s_u[lo], x = s_x[lo];
    ShGroup q;
    for (int g = lo * per;; ++g) {  // (the next border is past u)
      q = sh_group<S>(A, g);
      const uint32_t n = (uint32_t)q.units * q.tiles * A.n_kv;
      if (u - u0 < n) break;
      u0 += n, x += (uint32_t)(q.units ? q.tiles : 0) * A.n_kv;
    }
    q = {uni(q.row), uni(q.rows), uni(q.n), uni(q.tiles), uni(q.units)};
    u0 = (uint32_t)uni((int)u0), x = (uint32_t)uni((int)x);
    const uint32_t i = (u - u0) / in_place(q.units);
    const int kvh = i / in_place(q.tiles), ct = i - kvh * q.tiles, first = u - u0 - i * q.units;
    const int last = min((uint32_t)q.units, first + (u_end - u));  // units first .. last - 1 of the group's
    x += i;
    u += last - first;

    // the row that sees most of the shared positions, the first of those: its pages are read
    unsigned long long best = 0;
    for (int r = tid; r < q.rows; r += 256) {
      const unsigned long long v = (unsigned long long)min(sh_len(A, q.row + r), q.n) << 32 | (0xFFFFFFFFu - (uint32_t)r);
      best = v > best ? v : best;
    }
    for (int o = 32; o > 0; o >>= 1) {
      const unsigned long long v = __shfl_xor(best, o, 64);
      best = v > best ? v : best;
    }
    __syncthreads();  // (the previous piece is done with LDS)
    if (lane == 0) s_lead[w] = best;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) best = s_lead[k] > best ? s_lead[k] : best;
    const int reach = uni((int)(best >> 32));  // positions that some row sees
    const int lead = q.row + uni((int)(0xFFFFFFFFu - (uint32_t)best));
    const int units = min(last, (reach + S::STAGE - 1) / S::STAGE) - first;

    // this lane's columns
    int my_n[QT];
    uint4 qf[QT][G::NC];
    int n_min = 0x7FFFFFFF, n_max = 0;
#pragma unroll
    for (int y = 0; y < QT; ++y) {
      const int c = ct * COLS + (w * QT + y) * 16 + m16, r = c / A.heads, h = kvh * A.heads + (c - r * A.heads);
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

    // ---- staging: loads of 1 KB straight to LDS, three stages ahead ----
    constexpr int ROWS = 1024 / S::ROW;  // positions of a load
    const int32_t* tab = A.table + (int64_t)(reach > 0 ? uni(A.req ? ldg(A.req + lead) : lead) : 0) * A.table_stride;
    const int64_t head = (int64_t)kvh * A.head_stride * G::ES;
    const auto page_of = [&](int t) { return (int)(((uint64_t)(uint32_t)t * A.ps_mul) >> (31 + A.ps_shift)); };
    const auto row_of = [&](int j) { return (w + 4 * j) * ROWS + lane / S::PIECES; };  // of this lane's piece, load j
    const auto position = [&](int s) { return min((first + s) * S::STAGE + lane % S::STAGE, reach - 1); };
    const auto look_up = [&](int s) { return ldg(tab + page_of(position(min(s, units - 1)))); };
    // stage s, whose pages are `page` (a position a lane); returns those of its
    // positions that are on no page
    const auto load = [&](int s, int page) {
      const int t = position(s);
      const bool ok = page >= 0 && page < A.n_pages;
      const int64_t off =
          (ok ? (int64_t)page * A.page_stride + (int64_t)(t - page_of(t) * A.page_size) * A.token_stride : 0) * G::ES + head;
      char* to = s_kv[s % S::RING];
#pragma unroll
      for (int j = 0; j < S::LOADS; ++j) {
        const int row = row_of(j), at = 16 * sh_slot<S::ROW>(row, lane % S::PIECES);
        const uint32_t lo = __shfl((int)(uint32_t)off, row, 64), hi = __shfl((int)(off >> 32), row, 64);
        const int64_t o = (int64_t)((uint64_t)hi << 32 | lo) + (EXACT ? at : min(at, row_bytes - 16));
        __builtin_amdgcn_global_load_lds((const GLOBAL void*)((const char*)A.k + o), (lds_void*)(to + (w + 4 * j) * 1024), 16,
                                         0, 0);
        __builtin_amdgcn_global_load_lds((const GLOBAL void*)((const char*)A.v + o),
                                         (lds_void*)(to + S::BYTES + (w + 4 * j) * 1024), 16, 0, 0);
      }
      return (uint64_t)__ballot(!ok);
    };
    int page3 = 0, page4 = 0;                  // of stages s + 3, s + 4
    uint64_t away0 = 0, away1 = 0, away2 = 0;  // of stages s, s + 1, s + 2
    if (units > 0) {
      const int p0 = look_up(0), p1 = look_up(1), p2 = look_up(2);
      page3 = look_up(3), page4 = look_up(4);
      away0 = load(0, p0);
      if (units > 1) away1 = load(1, p1);
      if (units > 2) away2 = load(2, p2);
    }
    const uint32_t lds = (uint32_t)(uintptr_t)(lds_void*)&s_kv[0][0];
    const uint32_t k_at = m16 * S::ROW + 16 * sh_slot<S::ROW>(m16, gq);  // (chunk c: ^ 64 c, 16 positions on: + 16 ROW)
    uint32_t v_at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 4 * gq + j, b = m16 * G::VB;
      v_at[j] = S::BYTES + row * S::ROW + 16 * sh_slot<S::ROW>(row, b / 16) + b % 16;
    }
    for (int s = 0; s < units; ++s) {
      // this wave's part of stage s is there when those of the two behind it are
      // the only loads that are out; then all waves' parts are
      if (s + 2 < units)
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(4 * S::LOADS));
      else
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
      lds_barrier();
      const uint64_t away = away0;
      away0 = away1, away1 = away2;
      if (s + 3 < units) {
        const int page = page3;
        page3 = page4;
        page4 = look_up(s + 5);
        away2 = load(s + 3, page);
      }
      if (n_max == 0) continue;
#pragma unroll 1
      for (int tt = 0; tt < S::STAGE / TILE; ++tt) {
        const int t = (first + s) * S::STAGE + tt * TILE;
        if (t >= n_max) break;
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
        const uint32_t gone = (uint32_t)(away >> (tt * TILE)) & (uint32_t)((1ull << TILE) - 1);
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
                    uint32_t& v = tile.v[sb][j][ng][e];
                    const bool hi = (v & 0x7F800000u) == 0x7F800000u, lo = G::ES == 2 && (v & 0x7F80u) == 0x7F80u;
                    odd |= hi || lo;
                    v = G::ES == 4 ? (hi ? 0u : v) : (hi ? v & 0xFFFFu : v) & (lo ? 0xFFFF0000u : ~0u);
                  }
              }
            }
          odd = __any(odd);
        }
#pragma unroll
        for (int y = 0; y < QT; ++y) {
          float tm = sc[y][0][0];
#pragma unroll
          for (int sb = 0; sb < SUB; ++sb)
#pragma unroll
            for (int j = 0; j < 4; ++j) tm = fmaxf(tm, sc[y][sb][j]);
          // The reference of a column's powers of two moves where a score passes it
          // by 2^8: until then the powers stay far inside fp32, and nothing has to
          // cross lanes.
          if (__any(fmaf(tm, A.scale_log2, -mx[y]) > 8.f)) {
            const float mn = fmaxf(mx[y], max_over_rows(tm) * A.scale_log2);
            const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(mx[y] - mn);
            l[y] *= f;
#pragma unroll
            for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
              for (int e = 0; e < G::VD; ++e) acc[y][ng][e] *= f;
            mx[y] = mn;
          }
          const float ref = mx[y] == -INFINITY ? 0.f : mx[y];
#pragma unroll
          for (int sb = 0; sb < SUB; ++sb)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              sc[y][sb][j] = __builtin_amdgcn_exp2f(fmaf(sc[y][sb][j], A.scale_log2, -ref));
              l[y] += sc[y][sb][j];
            }
        }
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
                typedef uint32_t vec __attribute__((ext_vector_type(G::VB / 4)));
                const int b16 = (16 * ng + 4 * gq + r) * G::VB;  // (bytes of the row)
                const vec x4 = *(const vec*)(vp + p * S::ROW + 16 * sh_slot<S::ROW>(p, b16 / 16) + b16 % 16);
#pragma unroll
                for (int i = 0; i < G::VD; ++i) {
                  const float v = __uint_as_float(G::ES == 4 ? x4[i % (G::VB / 4)] : i & 1 ? x4[i / 2] & 0xFFFF0000u : x4[i / 2] << 16);
#pragma unroll
                  for (int y = 0; y < QT; ++y)
                    if (!isfinite(v) && t + p < my_n[y]) acc[y][ng][i][r] += v;
                }
              }
          }
        }
      }
    }

    // ---- the piece's sums to its slot ----
    float* out = A.seeds + (int64_t)(blockIdx.x + x) * COLS * (DP + 4);
#pragma unroll
    for (int y = 0; y < QT; ++y) {
      float sum = l[y];
      sum += __shfl_xor(sum, 16, 64);
      sum += __shfl_xor(sum, 32, 64);
      const int c = (w * QT + y) * 16 + m16;
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

template <typename T, int DP>
void sh_launch(const SharedArgs& A, int blocks, hipStream_t s) {
  if (A.head_dim == DP)
    hipLaunchKernelGGL((k_shared_prefix<T, DP, true>), dim3(blocks), dim3(256), 0, s, A);
  else
    hipLaunchKernelGGL((k_shared_prefix<T, DP, false>), dim3(blocks), dim3(256), 0, s, A);
}
template <typename T>
void sh_dim(const SharedArgs& A, int dp, int blocks, hipStream_t s) {
  if (dp == 64) sh_launch<T, 64>(A, blocks, s);
  else if (dp == 128) sh_launch<T, 128>(A, blocks, s);
  else sh_launch<T, 256>(A, blocks, s);
}

// columns of a work-group, positions of a unit
int sh_cols(int es, int dp) { return dp * es >= 1024 ? 64 : 128; }
int sh_blocks(int units) { return 2 * units; }
// (group, key head, tile)s of up to n_rows rows in up to n_groups groups
int64_t sh_tiles(int64_t n_rows, int64_t n_groups, int64_t group, int64_t n_kv, int cols) {
  return n_kv * (n_rows * group / cols + n_groups);
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
  const int es = dtype == SCUTE_F32 ? 4 : 2, dp = att_dim(head_dim), cols = sh_cols(es, dp);
  const int64_t slots = sh_blocks(units) + sh_tiles(max_rows, max_groups, n_heads / n_kv_heads, n_kv_heads, cols);
  const int64_t rows = ((int64_t)max_rows * sizeof(AttRowFrom) + 255) / 256 * 256;
  *bytes = (att_workspace(units, head_dim) + 255) / 256 * 256 + rows + slots * cols * (dp + 4) * 4;
  return SCUTE_OK;
}

extern "C" scute_status scute_shared_attention(const scute_kv_cache* C, const void* q, int64_t q_stride,
                                               int32_t n_heads, const int32_t* table, int64_t table_stride,
                                               int32_t n_requests, int32_t table_width, const int32_t* len,
                                               const int32_t* req, int32_t n_rows, const int32_t* group,
                                               const int32_t* shared_len, int32_t n_groups, float scale, void* out,
                                               int64_t out_stride, void* workspace, int64_t workspace_bytes,
                                               void* stream) {
  const char* fn = "scute_shared_attention";
  const auto bad = [&](scute_status code, const char* what) { return fail(code, std::string(fn) + ": " + what); };
  AttCall c{C, q, q_stride, n_heads, table, table_stride, n_requests, table_width, len, req, n_rows, scale,
            0, 0, out, out_stride, workspace, workspace_bytes, nullptr, nullptr, 1};
  scute_status st = att_check(fn, c);
  if (st != SCUTE_OK) return st;
  if (n_groups < 0 || n_groups > 65536) return bad(SCUTE_E_SHAPE, "n_groups must be in [0, 65536]");
  if (n_rows == 0) return SCUTE_OK;
  if (n_groups > 0 && (!group || !shared_len)) return bad(SCUTE_E_INVALID, "null pointer");
  if (((uintptr_t)group | (uintptr_t)shared_len) & 3) return bad(SCUTE_E_INVALID, "misaligned pointer");
  OnDevice g(C->device);
  if (!g.ok()) return hip_fail(g.err, fn);
  int64_t need = 0;
  if ((st = scute_shared_attention_workspace(C->device, C->dtype, C->head_dim, n_heads, C->n_kv_heads, n_rows, n_groups,
                                             &need)) != SCUTE_OK)
    return st;
  if (workspace_bytes < need) return bad(SCUTE_E_INVALID, "the workspace is too small");
  const int units = device_units(C->device), es = C->dtype == SCUTE_F32 ? 4 : 2, dp = att_dim(C->head_dim);
  const int group_heads = n_heads / C->n_kv_heads, cols = sh_cols(es, dp);
  const int64_t reach = std::min<int64_t>((int64_t)table_width * C->page_size, (int64_t)1 << 29);
  // (units are counted in 31 bits)
  const int64_t tiles = sh_tiles(n_rows, n_groups, group_heads, C->n_kv_heads, cols);
  if (tiles >= SH_TILES || tiles * (reach / sh_stage(es, dp) + 1) >= ((int64_t)1 << 31))
    return bad(SCUTE_E_SHAPE, "too many rows and heads for a table this wide");
  const int64_t own = (att_workspace(units, C->head_dim) + 255) / 256 * 256;
  char* ws = (char*)workspace;
  AttRowFrom* from = (AttRowFrom*)(ws + own);
  float* seeds = (float*)(ws + own + ((int64_t)n_rows * sizeof(AttRowFrom) + 255) / 256 * 256);
  int shift = 0;
  while ((1 << shift) < C->page_size) ++shift;
  const uint64_t mul = (((uint64_t)1 << (31 + shift)) + C->page_size - 1) / C->page_size;
  const SharedArgs A{q, C->k, C->v, table, len, req, group, shared_len, from, seeds, q_stride, C->page_stride,
                     C->token_stride, C->head_stride, table_stride, C->n_pages, (uint32_t)mul, n_rows, n_groups,
                     C->n_kv_heads, group_heads, C->head_dim, C->page_size, shift, (int32_t)reach, n_requests, (int32_t)tiles,
                     scale < 0.f, std::max(fabsf(scale * 1.4426950408889634f), 1e-37f)};
  const hipStream_t s = (hipStream_t)stream;
  if (es == 4) sh_dim<float>(A, dp, sh_blocks(units), s);
  else sh_dim<uint16_t>(A, dp, sh_blocks(units), s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e, fn);
  c.from = from, c.seeds = seeds, c.seed_cols = cols;
  return att_run(fn, c, ATT_SUFFIX, s);
}
