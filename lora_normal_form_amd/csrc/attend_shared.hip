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
  float scale_log2;
};

// Geometry of one instantiation.
template <typename T, int DP>
struct ShGeo {
  using G = AttGeo<T, DP>;
  static constexpr int QT = DP * G::ES >= 1024 ? 1 : 2;  // query tiles a wave (one where two would not fit the registers)
  static constexpr int COLS = 4 * 16 * QT;               // columns of a work-group
  static constexpr int ROW = DP * G::ES;                 // bytes of a position in LDS, without its padding
  static constexpr int STAGE = 16384 / ROW > 64 ? 64 : 16384 / ROW;  // positions staged at once: a unit
  static constexpr int PIECES = ROW / 16, PASS = STAGE * PIECES / 256;  // 16-byte pieces; passes of all threads
  static constexpr int PAD = ROW + 16;
};

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
__global__ __launch_bounds__(256) void k_shared_prefix(SharedArgs A) {
  using G = AttGeo<T, DP>;
  using S = ShGeo<T, DP>;
  constexpr int TILE = G::TILE, SUB = G::SUB, QT = S::QT, COLS = S::COLS;
  __shared__ __align__(16) char s_k[2][S::STAGE][S::PAD];
  __shared__ __align__(16) char s_v[2][S::STAGE][S::PAD];
  __shared__ uint32_t s_away[2][S::STAGE];  // positions whose page is outside the cache
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
        qf[y][k] = my_n[y] > 0 && (EXACT || at < row_bytes) ? v : make_uint4(0, 0, 0, 0);
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

    // ---- staging: this thread's piece of PASS positions a unit ----
    const int piece = tid % S::PIECES, p0 = tid / S::PIECES;
    constexpr int STEP = 256 / S::PIECES;
    const int req = A.req ? ldg(A.req + lead) : lead;
    const int32_t* tab = A.table + (int64_t)(reach > 0 ? uni(req) : 0) * A.table_stride;
    const int64_t head = (int64_t)kvh * A.head_stride * G::ES;
    const uint32_t at16 = EXACT ? 16 * piece : min(16 * piece, row_bytes - 16);
    const bool in_row = EXACT || 16 * piece < row_bytes;
    const auto page_of = [&](int t) { return (int)(((uint64_t)(uint32_t)t * A.ps_mul) >> (31 + A.ps_shift)); };
    int page[S::PASS];
    uint4 rk[S::PASS], rv[S::PASS];
    uint32_t away = 0;  // bit j: pass j's position has no page
    const auto look_up = [&](int s) {
#pragma unroll
      for (int j = 0; j < S::PASS; ++j)
        page[j] = ldg(tab + page_of(min((first + s) * S::STAGE + p0 + j * STEP, reach - 1)));
    };
    const auto load = [&](int s) {
      away = 0;
#pragma unroll
      for (int j = 0; j < S::PASS; ++j) {
        const int t = min((first + s) * S::STAGE + p0 + j * STEP, reach - 1);
        const bool ok = page[j] >= 0 && page[j] < A.n_pages;
        const int64_t off =
            (ok ? (int64_t)page[j] * A.page_stride + (int64_t)(t - page_of(t) * A.page_size) * A.token_stride : 0) * G::ES + head;
        rk[j] = ldg_b16<false>((const char*)A.k + off, at16);
        rv[j] = ldg_b16<false>((const char*)A.v + off, at16);
        away |= ok ? 0u : 1u << j;
      }
    };
    const auto put = [&](int b) {
#pragma unroll
      for (int j = 0; j < S::PASS; ++j) {
        const int p = p0 + j * STEP;
        const bool keep = in_row && !(away >> j & 1);
        *(uint4*)&s_k[b][p][16 * piece] = keep ? rk[j] : make_uint4(0, 0, 0, 0);
        *(uint4*)&s_v[b][p][16 * piece] = keep ? rv[j] : make_uint4(0, 0, 0, 0);
        if (piece == 0) s_away[b][p] = away >> j & 1;
      }
    };
    if (units > 0) {
      look_up(0);
      load(0);
      look_up(min(1, units - 1));
    }
    for (int s = 0; s < units; ++s) {
      const int b = s & 1;
      put(b);
      if (s + 1 < units) {
        load(s + 1);
        look_up(min(s + 2, units - 1));
      }
      __syncthreads();
      if (n_max == 0) continue;
#pragma unroll 1
      for (int tt = 0; tt < S::STAGE / TILE; ++tt) {
        const int t = (first + s) * S::STAGE + tt * TILE;
        if (t >= n_max) break;
        AttTile<T, DP, EXACT> tile;
        const char *kp = s_k[b][tt * TILE], *vp = s_v[b][tt * TILE];
#pragma unroll
        for (int sb = 0; sb < SUB; ++sb)
#pragma unroll
          for (int c = 0; c < G::NC; ++c) tile.k[sb][c] = *(const uint4*)(kp + (16 * sb + m16) * S::PAD + 64 * c + 16 * gq);
        f32x4 sc[QT][SUB];
        tile.template scores<QT>([&](int y, int c) { return qf[y][c]; }, sc, gq, row_bytes);
        const uint32_t gone = (uint32_t)__ballot(lane < TILE && s_away[b][tt * TILE + (lane & (TILE - 1))] != 0);
#pragma unroll
        for (int sb = 0; sb < SUB; ++sb)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int ng = 0; ng < G::NG; ++ng) {
              typedef uint32_t vec __attribute__((ext_vector_type(G::VB / 4)));
              const vec x4 = *(const vec*)(vp + (16 * sb + 4 * gq + j) * S::PAD + (16 * ng + m16) * G::VB);
#pragma unroll
              for (int e = 0; e < G::VB / 4; ++e) tile.v[sb][j][ng][e] = x4[e];
            }
#pragma unroll
        for (int y = 0; y < QT; ++y)
#pragma unroll
          for (int sb = 0; sb < SUB; ++sb) sc[y][sb] *= A.scale_log2;
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
                    const uint32_t v = tile.v[sb][j][ng][e];
                    odd |= (v & 0x7F800000u) == 0x7F800000u || (G::ES == 2 && (v & 0x7F80u) == 0x7F80u);
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
          const float mn = fmaxf(mx[y], max_over_quarters(tm));
          if (__any(mn > mx[y])) {
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
              sc[y][sb][j] = __builtin_amdgcn_exp2f(sc[y][sb][j] - ref);
              l[y] += sc[y][sb][j];
            }
        }
        if (!odd) {
          tile.template weigh<QT, false, true>(sc, acc);
        } else {  // a column after the other, with V cleared where it does not see it
          for (int c = 0; c < 16; ++c) {
#pragma unroll
            for (int y = 0; y < QT; ++y) {
              const int n = lane_of(my_n[y], c);
              uint32_t mask[SUB][4];
#pragma unroll
              for (int sb = 0; sb < SUB; ++sb)
#pragma unroll
                for (int j = 0; j < 4; ++j) mask[sb][j] = t + 16 * sb + 4 * gq + j >= n ? 0u : ~0u;
              f32x4 p1[1][SUB], a1[1][G::NG][G::VD];
#pragma unroll
              for (int sb = 0; sb < SUB; ++sb) p1[0][sb] = sc[y][sb];
#pragma unroll
              for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
                for (int e = 0; e < G::VD; ++e) a1[0][ng][e] = acc[y][ng][e];
              tile.template weigh<1, true, true>(p1, a1, mask, m16 == c);
#pragma unroll
              for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
                for (int e = 0; e < G::VD; ++e) acc[y][ng][e] = a1[0][ng][e];
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
int sh_stage(int es, int dp) { return std::min(64, 16384 / (dp * es)); }
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
                     scale * 1.4426950408889634f};
  const hipStream_t s = (hipStream_t)stream;
  if (es == 4) sh_dim<float>(A, dp, sh_blocks(units), s);
  else sh_dim<uint16_t>(A, dp, sh_blocks(units), s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_fail(e, fn);
  c.from = from, c.seeds = seeds, c.seed_cols = cols;
  return att_run(fn, c, ATT_SUFFIX, s);
}
