// The kernel of attention over the paged cache, for its forms (attend.hip,
// attend_sinks.hip), and its tiles' products (attend_shared.hip too).
#pragma once

#include <math.h>

#include <type_traits>

#include "block.h"
#include "kernels.h"

namespace scute {

// What a row's positions are:
//   ATT_PLAIN   the last `window` below its length (0: all)
//   ATT_SINKS   those, and the first `sinks`
enum : int { ATT_PLAIN = 0, ATT_SINKS = 1 };

struct AttArgs {
  const void *q, *k, *v;
  void* out;
  const int32_t *table, *len, *req;
  float* part;  // partial results, two pieces a slice
  int32_t* count;
  int64_t q_stride, out_stride, page_stride, token_stride, head_stride, table_stride, n_pages;
  int32_t row0;  // the launch's first row (a request's own number where req is null)
  uint32_t part_bytes, ps_mul;  // t / page_size = t ps_mul >> 31 + ps_shift
  int32_t n_rows, n_kv, q_tiles, group, together, head_dim, page_size, ps_shift, reach, n_requests, window;
  float scale_log2;  // scale log2(e): the softmax runs on powers of two
  int32_t sinks;     // ATT_SINKS
};

// out[h] = sum_t softmax_t(scale q[h] . K[t]) V[t] with a running maximum and
// sum: one pass over K and V, bound by their bytes (64 rows of 16384 positions,
// 32 query and 8 key heads of 128 elements: 655 us, 6.6 TB/s; a plain streaming
// read of as much reaches 6.4 TB/s, with non-temporal loads 7.1).
//
// How the work is cut. A unit is four tiles of positions, one for each wave (a
// tile: 32 of bf16, 16 of fp32), of one row, key head and tile of 16 query
// heads (32 where a key head has more than 16; or up to four rows of one
// request). Units are numbered row by row, key head by key head, and cut into
// slices of consecutive units, whatever rows and heads they cross: one slice a work-group, all alike, and where each has 64
// units or more a tail of short slices (1/16 of the units, 1/8 from 128 on) that
// the work-groups take from a counter as they get done: work-groups with equal
// work differ by a quarter in time, by their die and its distance to the memory
// (8 rows of 131072 positions: 758 us without the tail, 701 with; 2 of 100003,
// which have none: 145 with it, 135 without).
// Few rows whose heads come out even are cut along them instead (below). The
// figures of the cutting rules, here and below, are of 32 query and 8 key heads
// of 128 bf16 elements; other shapes follow the same rules without figures of
// their own.
// A slice's part of one (row, head) is a piece. A piece that holds all of its
// (row, head) writes the output; the others write partial results, and the
// last of them to arrive adds them in the pieces' order (where they are many the
// last of a group of 8 or more the group's first, then the last of all the
// groups'), so the result does not depend on who took which slice. Every
// work-group finds the slices from the lengths by itself (4 bytes a row), so
// nothing is planned on the host and a captured launch follows the lengths.
constexpr uint32_t ATT_EXTRA = 1;  // (128 ragged rows of up to 4096 positions: 190 us with 0, 181 with 1, 182 with 2)
// places of partial results a work-group: two a slice, at most 1 + 143 / 64
// slices a work-group and one more
constexpr int ATT_PLACES = 2 * 4, ATT_COLS = 32;  // (each of up to 32 columns)
// counters of the workspace: slices taken, work-groups done, and from
// ATT_ARRIVALS on the arrivals at each partial result's place, for groups of
// pieces and for all of them
constexpr int ATT_QUEUE = 0, ATT_DONE = 32, ATT_ARRIVALS = 64;

// Rows of one request that follow each other share its K and V: up to four of
// them (`together`, as many as fit the 16 columns of a query tile with all
// heads of a key head) are one row of the numbering, their first; the others
// have no units.
struct AttRow {
  int n, lo, first, units, req;     // positions some row sees: lo .. n - 1, in `units` units from tile `first`
  int rows, every_lo, every_n;      // rows, and the positions that each of them sees
  int sink;                         // ATT_SINKS: tiles from 0 on that come before tile `first`
};

// positions a row sees, from its length
__device__ __forceinline__ int att_len(const AttArgs& A, int len, int req) {
  return (uint32_t)req < (uint32_t)A.n_requests ? min(max(len, 0), A.reach) : 0;
}
// and the first of them (ATT_SINKS: behind the sinks)
__device__ __forceinline__ int att_first(const AttArgs& A, int n) {
  return A.window > 0 && n > A.window ? n - A.window : 0;
}
// whether a row whose positions begin at lo sees none at `at` (below its length)
template <int FORM>
__device__ __forceinline__ bool att_before(const AttArgs& A, int at, int lo) {
  return at < lo && !(FORM == ATT_SINKS && at < A.sinks);
}

template <int TILE, bool SHARED, int FORM>
__device__ __forceinline__ AttRow att_row(const AttArgs& A, int row) {
  AttRow r;
  bool leads = true;
  if (!SHARED || A.together == 1) {
    const int len = ldg(A.len + row);  // (asked for before req is known: one trip to memory, not two)
    r.req = A.req ? ldg(A.req + row) : A.row0 + row;
    r.n = att_len(A, len, r.req);
    r.lo = att_first(A, r.n);
    r.rows = 1, r.every_lo = r.lo, r.every_n = r.n;
  } else {
    const int base = row / A.together * A.together, me = row - base;
    int q[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = min(base + j, A.n_rows - 1);
      q[j] = ldg(A.req + at);
      l[j] = ldg(A.len + at);
    }
    const int own = me == 0 ? q[0] : me == 1 ? q[1] : me == 2 ? q[2] : q[3];
    leads = me == 0 || own != (me == 1 ? q[0] : me == 2 ? q[1] : q[2]);
    r.req = own, r.n = 0, r.lo = 0x7FFFFFFF, r.rows = 0, r.every_lo = 0, r.every_n = 0x7FFFFFFF;
    bool on = true;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      on = on && (j < me || (j < A.together && base + j < A.n_rows && q[j] == own));
      const int n = att_len(A, l[j], own), lo = att_first(A, n);
      if (on && j >= me) {
        r.n = max(r.n, n);
        if (n > 0) r.lo = min(r.lo, lo);
        r.every_lo = max(r.every_lo, lo);
        r.every_n = min(r.every_n, n);
        ++r.rows;
      }
    }
    r.lo = min(r.lo, r.n);
  }
  r.first = r.lo / TILE;
  r.sink = 0;
  if constexpr (FORM == ATT_SINKS) {
    r.sink = (min(A.sinks, r.lo) + TILE - 1) / TILE;
    if (r.sink >= r.first) r.sink = r.first = 0;  // (no tile between them)
  }
  r.units = max(1, ((r.n + TILE - 1) / TILE - r.first + r.sink + 3) >> 2);  // (an empty row writes its zeros)
  if (!leads) r.units = 0;
  return r;
}

__device__ __forceinline__ int lane_of(int v, int src) { return __builtin_amdgcn_readlane(v, src); }
// a uniform value that is computed with where it stands (a divisor whose
// reciprocal is not wanted ahead of the loop, on the way to the first loads)
__device__ __forceinline__ uint32_t in_place(uint32_t v) {
  asm volatile("" : "+s"(v));
  return v;
}
// inclusive sum over the wave's lanes, on row shifts and row broadcasts
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);
  return v;
}
__device__ __forceinline__ float max_over_quarters(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_frag(a), as_frag(b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma4(uint32_t a, uint32_t b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a), __uint_as_float(b), c, 0, 0, 0);
}
// ONCE: the bytes are read by this wave only (evicted first from the caches)
template <bool ONCE, typename V>
__device__ __forceinline__ V ldg_at(const char* p, uint32_t off) {
  if constexpr (ONCE)
    return __builtin_nontemporal_load((const GLOBAL V*)(p + off));
  else
    return *(const GLOBAL V*)(p + off);
}
template <bool ONCE>
__device__ __forceinline__ uint4 ldg_b16(const char* p, uint32_t off) {
  const u32x4 v = ldg_at<ONCE, u32x4>(p, off);
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ uint32_t dword(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Geometry of one instantiation: heads of up to DP elements of type T.
template <typename T, int DP>
struct AttGeo {
  static constexpr int ES = sizeof(T);
  static constexpr int SUB = ES == 2 ? 2 : 1;   // blocks of 16 positions in a tile
  static constexpr int TILE = 16 * SUB;
  static constexpr int NC = DP * ES / 64;       // 64-byte chunks of a K row
  static constexpr int VB = ES == 2 && DP == 64 ? 8 : 16;  // bytes of a V row a lane loads at once
  static constexpr int VD = VB / ES;            // elements of them
  static constexpr int NG = DP / (16 * VD);     // loads that cover a V row over 16 lanes
};

// One tile's products. Scores: S^T = K Q^T, K rows as the A operand (lane
// (m, g): row m of 16, the 16 bytes g of every 64-byte chunk; Q is laid out
// alike, so the order of the contraction does not matter), so a lane holds
// query m and positions 4 g + 0..3 of each 16. Output: O^T = V^T P^T with the
// contraction index permuted so that a lane's own scores are its P operand
// (nothing crosses lanes); V is loaded in rows, VD elements of rows
// 4 g + 0..3 per lane, and the V^T operand of element i is a permutation of
// bytes inside the lane. Output rows (dims) of lane (m, g), element i of load
// ng, register r: 16 VD ng + VD (4 g + r) + i; its column is query m again,
// so the softmax factors need no exchange either.
template <typename T, int DP, bool EXACT>
struct AttTile {
  using G = AttGeo<T, DP>;
  uint4 k[G::SUB][G::NC];
  uint32_t v[G::SUB][4][G::NG][G::VB / 4];

  template <bool ONCE>
  __device__ __forceinline__ void load_v(const char* p, uint32_t off, int s, int j, int ng) {
    typedef uint32_t vec __attribute__((ext_vector_type(G::VB / 4)));
    const vec x = ldg_at<ONCE, vec>(p, off);
#pragma unroll
    for (int e = 0; e < G::VB / 4; ++e) v[s][j][ng][e] = x[e];
  }
  // q(y, c): chunk c of query tile y
  template <int QT, typename Q>
  __device__ __forceinline__ void scores(const Q& q, f32x4 (&sc)[QT][G::SUB], int gq, int row_bytes) {
#pragma unroll
    for (int s = 0; s < G::SUB; ++s) {
#pragma unroll
      for (int y = 0; y < QT; ++y) sc[y][s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < G::NC; ++c) {
        if (!EXACT && DP > 64 && 64 * c >= row_bytes) continue;  // (uniform)
        uint4 kk = k[s][c];
        if constexpr (!EXACT)  // past the head's end: other elements, which may hold anything
          if (64 * c + 16 * gq >= row_bytes) kk = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int y = 0; y < QT; ++y) {
          if constexpr (G::ES == 2) {
            sc[y][s] = mfma16(kk, q(y, c), sc[y][s]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[y][s] = mfma4(dword(kk, e), dword(q(y, c), e), sc[y][s]);
          }
        }
      }
    }
  }
  __device__ __forceinline__ void clear_v(int s, int j) {
#pragma unroll
    for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
      for (int e = 0; e < G::VB / 4; ++e) v[s][j][ng][e] = 0;
  }
  // a tile's weights as operands
  template <int QT>
  struct Weights {
    uint4 b[QT], b2[G::ES == 2 ? QT : 1];
  };
  // bf16: the weights as sums of two bf16 (one alone would add an error of the
  // output's own rounding, 2^-8; the second products cost no time). The second is 0
  // or of either sign, so an infinite V gives a sum of any kind, which is put right
  // where the waves' results are joined. POS: both parts are positive (the first cut
  // off instead of rounded, the second 2^-20 of the weight more than the rest), so
  // that an infinite V stays infinite; the weight is off by 2^-15 at most.
  template <int QT, bool POS = false>
  static __device__ __forceinline__ Weights<QT> pack(const f32x4 (&p)[QT][G::SUB]) {
    Weights<QT> W;
    if constexpr (G::ES == 2) {
      const auto first = [](float x, float y) {
        return POS ? __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u)
                   : pack_bf2(__float_as_uint(x), __float_as_uint(y));
      };
      const auto rest = [](uint32_t hi, float x, float y) {
        if constexpr (POS)
          return pack_bf2(__float_as_uint(fmaf(x, 1.f + 0x1p-20f, -__uint_as_float(hi << 16))),
                          __float_as_uint(fmaf(y, 1.f + 0x1p-20f, -__uint_as_float(hi & 0xFFFF0000u))));
        return pack_bf2(__float_as_uint(x - __uint_as_float(hi << 16)), __float_as_uint(y - __uint_as_float(hi & 0xFFFF0000u)));
      };
#pragma unroll
      for (int y = 0; y < QT; ++y) {
        W.b[y].x = first(p[y][0][0], p[y][0][1]);
        W.b[y].y = first(p[y][0][2], p[y][0][3]);
        W.b[y].z = first(p[y][1][0], p[y][1][1]);
        W.b[y].w = first(p[y][1][2], p[y][1][3]);
        W.b2[y].x = rest(W.b[y].x, p[y][0][0], p[y][0][1]);
        W.b2[y].y = rest(W.b[y].y, p[y][0][2], p[y][0][3]);
        W.b2[y].z = rest(W.b[y].z, p[y][1][0], p[y][1][1]);
        W.b2[y].w = rest(W.b[y].w, p[y][1][2], p[y][1][3]);
      }
    } else {
#pragma unroll
      for (int y = 0; y < QT; ++y)
        W.b[y] = make_uint4(__float_as_uint(p[y][0][0]), __float_as_uint(p[y][0][1]), __float_as_uint(p[y][0][2]),
                            __float_as_uint(p[y][0][3]));
    }
    return W;
  }
  // V times them. SOME: of the positions that `mask` (ones or zeros for each) leaves,
  // for the columns of the lanes that `keep`
  template <int QT, bool SOME = false>
  __device__ __forceinline__ void products(const Weights<QT>& W, f32x4 (&acc)[QT][G::NG][G::VD],
                                           const uint32_t (*mask)[4] = nullptr, bool keep = true) {
    const auto val = [&](int s, int j, int ng, int i) { return SOME ? v[s][j][ng][i] & mask[s][j] : v[s][j][ng][i]; };
    const auto put = [&](f32x4& to, f32x4 x) {
#pragma unroll
      for (int r = 0; r < 4; ++r) to[r] = !SOME || keep ? x[r] : to[r];
    };
#pragma unroll
    for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
      for (int i = 0; i < G::VD; ++i) {
        if constexpr (G::ES == 2) {
          const uint32_t sel = i & 1 ? 0x07060302u : 0x05040100u;
          uint4 a;
          a.x = __builtin_amdgcn_perm(val(0, 1, ng, i / 2), val(0, 0, ng, i / 2), sel);
          a.y = __builtin_amdgcn_perm(val(0, 3, ng, i / 2), val(0, 2, ng, i / 2), sel);
          a.z = __builtin_amdgcn_perm(val(1, 1, ng, i / 2), val(1, 0, ng, i / 2), sel);
          a.w = __builtin_amdgcn_perm(val(1, 3, ng, i / 2), val(1, 2, ng, i / 2), sel);
#pragma unroll
          for (int y = 0; y < QT; ++y) put(acc[y][ng][i], mfma16(a, W.b2[y], mfma16(a, W.b[y], acc[y][ng][i])));
        } else {
#pragma unroll
          for (int y = 0; y < QT; ++y) {
            f32x4 x = acc[y][ng][i];
#pragma unroll
            for (int j = 0; j < 4; ++j) x = mfma4(val(0, j, ng, i), dword(W.b[y], j), x);
            put(acc[y][ng][i], x);
          }
        }
      }
  }
  template <int QT, bool SOME = false, bool POS = false>
  __device__ __forceinline__ void weigh(const f32x4 (&p)[QT][G::SUB], f32x4 (&acc)[QT][G::NG][G::VD],
                                        const uint32_t (*mask)[4] = nullptr, bool keep = true) {
    products<QT, SOME>(pack<QT, POS>(p), acc, mask, keep);
  }
};

// PAGE16: pages hold multiples of 16 positions, so the 16 of a block lie in
// one page and their place is one scalar; else every position is looked up.
// EXACT: the head dimension is DP. MODE:
//   ATT_ONCE    no two rows or query tiles read the same positions, so K and V
//               are loaded past the caches (2 rows of 100003 positions: 157 us
//               without, 141 with; rows that share positions lose: four drafted
//               tokens a request 39 us without, 48 with)
//   ATT_SHARED  rows of one request that follow each other are one query tile
//   ATT_WIDE    two query tiles at once, for more than 16 query heads a key head
enum : int { ATT_ONCE = 0, ATT_SHARED = 1, ATT_WIDE = 2 };
// One work-group a compute unit: four waves with a tile of K and V each in
// flight (64 KB at 128 elements) already fill the memory's queues, and fewer
// streams at once run faster than more (64 rows of 16384 positions: 674 us
// with one, 712 with two).
template <typename T, int DP, bool PAGE16, bool EXACT, int MODE, int FORM>
__global__ __launch_bounds__(256) void k_paged_attention(AttArgs A) {
  using G = AttGeo<T, DP>;
  constexpr int TILE = G::TILE, SUB = G::SUB, OS = DP + 4, QT = MODE == ATT_WIDE ? 2 : 1, COLS = 16 * QT;
  constexpr bool ONCE = MODE == ATT_ONCE, SHARED = MODE == ATT_SHARED;
  __shared__ float s_ml[4][COLS][2];
  __shared__ __align__(16) float s_o[4][COLS][OS];
  // The queries stay in LDS where the registers would not hold them too (23 rows
  // of 33324 positions, 18 heads of 176 over one: 301 us without, 130 with; where
  // they fit they are faster there: 64 rows of up to 2000, fp32, 48 heads of 128
  // over two: 64 us, 70 from LDS).
  constexpr bool Q_LDS = DP == 256 && QT * G::ES > 2;
  constexpr int QROW = DP * G::ES + 16;
  __shared__ __align__(16) char s_q[Q_LDS ? COLS * QROW : 16];
  __shared__ uint32_t s_wsum[4], s_before;
  __shared__ uint32_t s_next;
  __shared__ int s_row, s_last;
  const int tid = threadIdx.x, lane = tid & 63, w = uni(tid >> 6), m16 = lane & 15, gq = lane >> 4;
  const int H = A.n_kv * A.q_tiles, D = EXACT ? DP : A.head_dim, row_bytes = D * G::ES;

  // Units (all below 2^31: the host cuts the rows into launches for that) and
  // where the rows' begin. Up to 64 rows: a row a lane, every wave for itself.
  // Where (row, head)s are more than work-groups, each counts `extra` units
  // more than it has, in front of its own, for what a piece costs beside them.
  const uint32_t extra = (uint32_t)A.n_rows * H > gridDim.x * A.together ? ATT_EXTRA : 0;
  const auto cost = [&](const AttRow& r) { return r.units ? (uint32_t)r.units + extra : 0u; };
  const bool few = A.n_rows <= 64;
  AttRow mine = {};
  const int per = (A.n_rows + 255) / 256, r0 = min(A.n_rows, tid * per), r1 = min(A.n_rows, r0 + per);
  uint32_t own = 0, upto;  // units of one head: of this lane's rows, and up to them
  uint32_t U;
  if (few) {
    if (lane < A.n_rows) mine = att_row<TILE, SHARED, FORM>(A, lane);
    upto = wave_scan(cost(mine));
    U = (uint32_t)lane_of((int)upto, 63) * H;
  } else {
    for (int r = r0; r < r1; ++r) own += cost(att_row<TILE, SHARED, FORM>(A, r));
    upto = wave_scan(own);
    if (lane == 63) s_wsum[w] = upto;
    __syncthreads();
    U = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (x < w) upto += s_wsum[x];
      U += s_wsum[x];
    }
    U = (uint32_t)uni((int)U) * H;
  }
  const uint32_t workers = min(U, gridDim.x), each = U / workers;
  // Even pieces: no slice crosses from one (row, head) to the next, each of them
  // cut into parts of at most `most` units, one a work-group. Taken where that
  // costs at most one unit more than equal ranges: it saves the second piece of
  // the ranges that cross (16 requests of four drafted rows, up to 3000
  // positions: 36 us with ranges, 26 with parts; 2 rows of 100003: 133, 130;
  // with up to four units more 8 ragged rows of up to 16000 lose: 64, 67).
  bool even = false;
  uint32_t parts = 0, parts_upto = 0, even_slices = 0;  // parts of this lane's row, and up to it
  if (few && extra == 0 && each < 64) {
    uint32_t most = (U + gridDim.x - 1) / gridDim.x;
    for (int i = 0; i < 2 && !even; ++i, ++most) {
      parts = ((uint32_t)mine.units + most - 1) / in_place(most);
      // (two units stay whole: joining parts costs 1.4 us, a second trip 1 us)
      if (mine.units == 2) parts = 1;
      parts_upto = wave_scan(parts);
      even_slices = (uint32_t)lane_of((int)parts_upto, 63) * H;
      even = even_slices <= gridDim.x;
    }
  }
  // slices: `workers` of quot or quot + 1 units (the first `longer`), then from
  // unit `fixed` on of `step` units each
  const uint32_t tail = each >= 128 ? U / 8 : each >= 64 ? U / 16 : 0, step = max(4u, each / 16);
  const uint32_t fixed = U - tail, quot = tail ? fixed / workers : each, longer = fixed - quot * workers;
  const uint32_t slices = even ? even_slices : workers + (tail ? (tail + step - 1) / step : 0);
  const auto slice_of = [&](uint32_t unit) {  // the slice that holds a unit
    const uint32_t edge = longer * (quot + 1);
    if (unit >= fixed) return workers + (unit - fixed) / in_place(step);
    return unit < edge ? unit / in_place(quot + 1) : longer + (unit - edge) / in_place(quot);
  };
  const auto slice_begin = [&](uint32_t i) {
    return i < workers ? i * quot + min(i, longer) : min(U, fixed + (i - workers) * step);
  };
  const rsrc_t part = make_rsrc(A.part, A.part_bytes);
  constexpr uint32_t SLOT = COLS * (DP + 4) * 4;  // bytes of a partial result: COLS x (DP values, m, l, a group's m, l)

  uint32_t slice = blockIdx.x, u_begin = 0, u = 0, u_end = 0, base = 0;
  int row = 0;
  if (slice >= slices) return;
  bool asked = true;  // `slice` is new
  for (;;) {
    if (even) {
      row = (int)__popcll(__ballot(parts_upto * H <= slice));
    } else if (u == u_end) {  // the slice's units, the row they begin in and that row's first unit
      if (!asked) {
        if (tail && tid == 0) s_next = workers + (uint32_t)arrive(A.count + ATT_QUEUE);
        __syncthreads();
        slice = tail ? (uint32_t)uni((int)s_next) : slices;
        __syncthreads();
      }
      asked = false;
      if (slice >= slices) break;
      u = u_begin = slice_begin(slice);
      u_end = slice_begin(slice + 1);
      if (few) {
        row = (int)__popcll(__ballot(upto * H <= u));  // (rows that end before: their lanes come first)
        base = row ? (uint32_t)lane_of((int)upto, row - 1) * H : 0;
      } else {
        uint32_t pre = upto - own;
        if (pre * H <= u && u < upto * H) {
          int r = r0;
          for (uint32_t t = cost(att_row<TILE, SHARED, FORM>(A, r)); (pre + t) * H <= u; t = cost(att_row<TILE, SHARED, FORM>(A, r))) {
            pre += t;
            ++r;
          }
          s_row = r;
          s_before = pre;
        }
        __syncthreads();
        row = uni(s_row);
        base = (uint32_t)uni((int)s_before) * H;
      }
    }
    AttRow R;
    for (;; ++row) {  // (rows without units are passed)
      if (few) {
        R = {lane_of(mine.n, row), lane_of(mine.lo, row), lane_of(mine.first, row), lane_of(mine.units, row),
             lane_of(mine.req, row), 1, 0, 0, FORM == ATT_SINKS ? lane_of(mine.sink, row) : 0};
        if constexpr (SHARED)
          R.rows = lane_of(mine.rows, row), R.every_lo = lane_of(mine.every_lo, row), R.every_n = lane_of(mine.every_n, row);
      } else {
        R = att_row<TILE, SHARED, FORM>(A, row);
        R = {uni(R.n), uni(R.lo), uni(R.first), uni(R.units), uni(R.req), uni(R.rows), uni(R.every_lo), uni(R.every_n),
             FORM == ATT_SINKS ? uni(R.sink) : 0};
      }
      if (!SHARED || R.units) break;
    }
    if constexpr (!SHARED) R.every_lo = R.lo, R.every_n = R.n;
    // head and units of the piece, and (all) the pieces of its (row, head): one in
    // each of the slices w0 on, in the slice's first place but perhaps in w0
    uint32_t hh, v0, units, taken = 0, w0 = 0, all = 0, slot0 = 0;
    const uint32_t whole_cost = R.units + extra;
    if (even) {
      const uint32_t n = (uint32_t)lane_of((int)parts, row);
      const uint32_t x = slice - (row ? (uint32_t)lane_of((int)parts_upto, row - 1) * H : 0);
      hh = x / in_place(n);
      const uint32_t j = x - hh * n;
      v0 = j * R.units / in_place(n), units = (j + 1) * R.units / in_place(n) - v0;
      w0 = slice - j, all = n, slot0 = 2 * w0;
    } else {
      hh = (u - base) / in_place(whole_cost);
      const uint32_t x0 = u - base - hh * whole_cost;
      taken = min(whole_cost - x0, u_end - u);
      v0 = max(x0, extra) - extra, units = max(x0 + taken, extra) - extra - v0;
      if (units == 0) {  // (only what the piece counts beside its own)
        u += taken;
        continue;
      }
      if (units != (uint32_t)R.units) {
        const uint32_t a = u - x0;
        w0 = slice_of(a + extra), all = slice_of(a + whole_cost - 1) - w0 + 1;
        slot0 = 2 * w0 + (slice_begin(w0) >= a ? 0 : 1);
      }
    }
    // the piece's tiles of the row: t0 .. t0 + cnt - 1 from the row's first (its
    // sinks' tiles, then those from R.first on)
    const int t0 = 4 * (int)v0, cnt = min(4 * (int)units, (R.n + TILE - 1) / TILE - R.first + R.sink - t0);
    const int kvh = A.q_tiles == 1 ? hh : hh / in_place(A.q_tiles), h0 = kvh * A.group + (hh - kvh * A.q_tiles) * COLS;
    // columns of the query tile: column c is head h0 + c % wide of row c / wide
    const bool shared = SHARED && A.together > 1;
    const int wide = shared ? A.group : COLS, nq = shared ? R.rows * A.group : min(COLS, (kvh + 1) * A.group - h0);
    const int my_row = !SHARED ? 0 : min(m16, nq - 1) / in_place(wide);
    int my_n = R.n, my_lo = R.lo;  // what this lane's column sees
    if (shared && R.rows > 1) {
      my_n = att_len(A, ldg(A.len + row + my_row), R.req);
      my_lo = att_first(A, my_n);
    }

    // ---- the wave's tiles t0 + w, t0 + w + 4, ... ----
    float mx[QT], l[QT];
    f32x4 acc[QT][G::NG][G::VD];
#pragma unroll
    for (int y = 0; y < QT; ++y) {
      mx[y] = -INFINITY, l[y] = 0.f;
#pragma unroll
      for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
        for (int i = 0; i < G::VD; ++i) acc[y][ng][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // 16 bytes of a column of the query tile, zeros past its end
    const auto query = [&](int col, int of_row, int at) {
      const char* qp = (const char*)A.q + ((int64_t)(row + of_row) * A.q_stride + (int64_t)(h0 + min(col, nq - 1) - of_row * wide) * D) * G::ES;
      const uint4 x = ldg_b16<false>(qp, EXACT ? at : min(at, row_bytes - 16));
      return col < nq && (EXACT || at < row_bytes) ? x : make_uint4(0, 0, 0, 0);
    };
    if constexpr (Q_LDS) {
      for (int i = tid; i < COLS * G::NC * 4; i += 256) {
        const int col = i / (G::NC * 4), at = 16 * (i % (G::NC * 4));
        *(uint4*)&s_q[col * QROW + at] = query(col, SHARED ? min(col, nq - 1) / in_place(wide) : 0, at);
      }
      __syncthreads();
    }
    if (w < cnt) {  // (an empty row has none)
      const char *kb = (const char*)A.k, *vb = (const char*)A.v;
      const int32_t* tab = A.table + (int64_t)R.req * A.table_stride;
      const int64_t head = (int64_t)kvh * A.head_stride * G::ES;
      const uint32_t tok = (uint32_t)A.token_stride * G::ES;
      const int trips = (cnt - w + 3) >> 2, tb = (FORM == ATT_SINKS ? 0 : R.first) + t0 + w;  // tile of trip i: tb + 4 i
      const auto first_of = [&](int i) {  // the trip's first position
        const int x = tb + 4 * i;
        return (FORM == ATT_SINKS && x >= R.sink ? x - R.sink + R.first : x) * TILE;
      };
      const auto page_of = [&](int t) { return (int)(((uint64_t)(uint32_t)t * A.ps_mul) >> (31 + A.ps_shift)); };

      AttTile<T, DP, EXACT> tile;
      // places of the next 64 trips' blocks, a trip a lane (PAGE16): bytes from
      // k and v, -1 for a page outside the cache
      int32_t place_lo[SUB], place_hi[SUB];
      // the next trip's pages, a position of each block a lane (otherwise)
      int32_t page_next[SUB];
      const auto look_up = [&](int i) {
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
          if constexpr (PAGE16) {
            const int t = min(first_of(i + lane) + 16 * s, (R.n - 1) & ~15);
            const int at = page_of(t), page = ldg(tab + at);
            const int64_t off = ((int64_t)page * A.page_stride + (int64_t)(t - at * A.page_size) * A.token_stride) * G::ES + head;
            const bool ok = page >= 0 && page < A.n_pages;
            place_lo[s] = ok ? (int32_t)(uint32_t)off : -1;
            place_hi[s] = ok ? (int32_t)(off >> 32) : -1;
          } else {
            const int t = min(first_of(i) + 16 * s + m16, R.n - 1);
            page_next[s] = ldg(tab + page_of(t));
          }
        }
      };
      int64_t off[SUB];       // PAGE16: of the block; else of this lane's position m16
      uint32_t bad[SUB];      // bits of the positions whose page is outside the cache
      const auto locate = [&](int i) {
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
          if constexpr (PAGE16) {
            const int src = i & 63;
            const int64_t o = (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readlane(place_hi[s], src) << 32) |
                                        (uint32_t)__builtin_amdgcn_readlane(place_lo[s], src));
            bad[s] = o < 0 ? 0xFFFFu : 0u;
            off[s] = o < 0 ? head : o;
          } else {
            const int t = min(first_of(i) + 16 * s + m16, R.n - 1), page = page_next[s];
            const bool ok = page >= 0 && page < A.n_pages;
            off[s] = (ok ? ((int64_t)page * A.page_stride + (int64_t)(t - page_of(t) * A.page_size) * A.token_stride) * G::ES
                         : 0) + head;
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
            tile.k[s][c] = ldg_b16<ONCE>(kb + off[s], PAGE16 ? m16 * tok + at : at);
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
              const uint32_t lo = __shfl((int)(uint32_t)off[s], src, 64), hi = __shfl((int)(off[s] >> 32), src, 64);
              p = vb + (int64_t)(((uint64_t)hi << 32) | lo);
              o = 0;
            }
#pragma unroll
            for (int ng = 0; ng < G::NG; ++ng) {
              const int at = (16 * ng + m16) * G::VB;
              tile.template load_v<ONCE>(p, o + (EXACT ? at : min(at, row_bytes - G::VB)), s, j, ng);
            }
          }
      };

      look_up(0);
      uint4 q[Q_LDS ? 1 : QT][G::NC];
      if constexpr (!Q_LDS) {
#pragma unroll
        for (int y = 0; y < QT; ++y)
#pragma unroll
          for (int c = 0; c < G::NC; ++c) q[y][c] = query(16 * y + m16, my_row, 64 * c + 16 * gq);
      }
      locate(0);
      load_k();
      load_v();
      if constexpr (!PAGE16) look_up(min(1, trips - 1));
      // (the loads of trip i + 1 run under the products of trip i; the last trip
      // stands apart, so that the waits count what is in flight)
      const auto trip = [&](int i, auto more) {
        const int t = first_of(i);
        uint32_t gone[SUB];
        bool cut = t < R.every_lo || t + TILE > R.every_n;
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
          gone[s] = bad[s];
          cut = cut || bad[s] != 0;
        }
        f32x4 sc[QT][SUB];
        if constexpr (Q_LDS) {
          const char* qp = &s_q[m16 * QROW + 16 * gq + (int)in_place(0)];  // (read in every trip, not kept)
          tile.template scores<QT>([&](int y, int c) { return *(const uint4*)(qp + 16 * y * QROW + 64 * c); }, sc, gq, row_bytes);
        } else {
          tile.template scores<QT>([&](int y, int c) { return q[y][c]; }, sc, gq, row_bytes);
        }
        if constexpr (more) {
          if constexpr (PAGE16) {
            if (((i + 1) & 63) == 0) look_up(i + 1);
          }
          locate(i + 1);
          load_k();
          if constexpr (!PAGE16) look_up(min(i + 2, trips - 1));
        }
#pragma unroll
        for (int y = 0; y < QT; ++y)
#pragma unroll
          for (int s = 0; s < SUB; ++s) sc[y][s] *= A.scale_log2;
        const auto each_place = [&](auto f) {  // f(block, position of it, position, whether its page is not there)
#pragma unroll
          for (int s = 0; s < SUB; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) f(s, j, t + 16 * s + 4 * gq + j, (gone[s] >> (4 * gq + j)) & 1);
        };
        // a position that is not seen has no weight, and its value, which may be
        // anything, is cleared
        if (cut) {
          each_place([&](int s, int j, int at, bool away) {
            if (att_before<FORM>(A, at, my_lo) || at >= my_n || away) {
#pragma unroll
              for (int y = 0; y < QT; ++y) sc[y][s][j] = -INFINITY;
            }
          });
          if (!SHARED || R.rows == 1)
            each_place([&](int s, int j, int at, bool away) {
              if (att_before<FORM>(A, at, R.lo) || at >= R.n || away) tile.clear_v(s, j);
            });
        }
#pragma unroll
        for (int y = 0; y < QT; ++y) {
          float tm = sc[y][0][0];
#pragma unroll
          for (int s = 0; s < SUB; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) tm = fmaxf(tm, sc[y][s][j]);
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
          for (int s = 0; s < SUB; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              sc[y][s][j] = __builtin_amdgcn_exp2f(sc[y][s][j] - ref);
              l[y] += sc[y][s][j];
            }
        }
        if (!SHARED || !cut || R.rows == 1) {
          tile.template weigh<QT>(sc, acc);
        } else {
          // rows that see different parts of the tile: each on its own, with V
          // cleared for it (what others see of it, times their weight of 0, may
          // be NaN: only the row's own columns are kept). V is masked as it is
          // used: with copies of V and of the sums heads of more than 128 elements
          // left the registers (136 requests of five rows over 1895 positions, 11
          // heads of 240 over one: 472 us with copies, 200 without).
          for (int i = 0; i < R.rows; ++i) {
            const int lo = lane_of(my_lo, i * wide), n = lane_of(my_n, i * wide);
            uint32_t mask[SUB][4];
            each_place([&](int s, int j, int at, bool away) { mask[s][j] = att_before<FORM>(A, at, lo) || at >= n || away ? 0u : ~0u; });
            tile.template weigh<QT, true>(sc, acc, mask, my_row == i);
          }
        }
        if constexpr (more) load_v();
      };
      for (int i = 0; i + 1 < trips; ++i) trip(i, std::true_type());
      trip(trips - 1, std::false_type());
    }
#pragma unroll
    for (int y = 0; y < QT; ++y) {
      l[y] += __shfl_xor(l[y], 16, 64);
      l[y] += __shfl_xor(l[y], 32, 64);
    }
    // the next slice, asked for while the results are joined
    const bool last_piece = !even && u + taken == u_end;
    uint32_t next = slices;
    if (last_piece && tail && tid == 0) next = workers + (uint32_t)arrive(A.count + ATT_QUEUE);

    // ---- the four waves' results joined in LDS ----
    const int waves = max(0, min(cnt, 4));  // those with tiles
#pragma unroll
    for (int y = 0; y < QT; ++y) {
      const int col = 16 * y + m16;
      if (w < waves && col < nq) {
        if (gq == 0) s_ml[w][col][0] = mx[y], s_ml[w][col][1] = l[y];
#pragma unroll
        for (int ng = 0; ng < G::NG; ++ng)
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < G::VD; i += 4)
              *(f32x4*)&s_o[w][col][16 * G::VD * ng + G::VD * (4 * gq + r) + i] =
                  f32x4{acc[y][ng][i][r], acc[y][ng][i + 1][r], acc[y][ng][i + 2][r], acc[y][ng][i + 3][r]};
      }
    }
    __syncthreads();
    const bool whole = units == (uint32_t)R.units;
    const int E = nq * D / 4;  // groups of four elements of the piece's output
    const auto put = [&](int g, int d, f32x4 o, float L) {
      const f32x4 x = L == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : o / L;
      const int i = !SHARED ? 0 : g / wide;
      const int64_t at = (int64_t)(row + i) * A.out_stride + (int64_t)(h0 + g - i * wide) * D + d;
      if constexpr (G::ES == 4) {
        stg4((float*)A.out + at, x);
      } else {
        typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
        *(GLOBAL u32x2*)((uint16_t*)A.out + at) = u32x2{pack_bf2(__float_as_uint(x.x), __float_as_uint(x.y)),
                                                       pack_bf2(__float_as_uint(x.z), __float_as_uint(x.w))};
      }
    };
    const uint32_t slot = 2 * slice + (even || u == u_begin ? 0 : 1);
    for (int e = tid; e < E; e += 256) {
      const int g = e / (D / 4), d = 4 * (e - g * (D / 4));
      float gm = -INFINITY, L = 0.f, wm[4], wl[4];
      f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f}, wo[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {  // (all four waves' at once; what a wave without tiles left there is not used)
        wm[x] = s_ml[x][g][0], wl[x] = s_ml[x][g][1];
        wo[x] = *(const f32x4*)&s_o[x][g][d];
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        wm[x] = x < waves ? wm[x] : -INFINITY;
        gm = fmaxf(gm, wm[x]);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float f = gm == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(wm[x] - gm);
        if (x < waves) L += wl[x] * f, o += wo[x] * f;
      }
      if constexpr (G::ES == 2) {
        // Not finite, beside weights whose sum is: some V that the column sees is
        // not finite. These elements are the sum of what is not finite there,
        // whatever the (positive) weights: the piece's positions are gone through
        // once more for it (four loads in flight: with eight the 32 columns of 256
        // elements spilled in their main loop, 64 rows of 3000 positions, 24 heads
        // over one: 61 us with four, 69 with eight).
        if (__builtin_expect(fmaf(o.x, 0.f, fmaf(o.y, 0.f, fmaf(o.z, 0.f, o.w * 0.f))) != 0.f && isfinite(L), 0)) {
          typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
          const int i = SHARED ? g / wide : 0;
          const int n = shared ? att_len(A, ldg(A.len + row + i), R.req) : R.n;
          const int lo = att_first(A, n);
          const int32_t* tab = A.table + (int64_t)R.req * A.table_stride;
          const char* vp = (const char*)A.v + ((int64_t)kvh * A.head_stride + d) * G::ES;
          f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
          const auto look = [&](int from, int to) {
            for (int t = from; t < to; t += 4) {
              uint2 v[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int at = min(t + x, to - 1), p = (int)(((uint64_t)(uint32_t)at * A.ps_mul) >> (31 + A.ps_shift));
                const int page = ldg(tab + p);
                const bool seen = t + x < to && page >= 0 && page < A.n_pages;
                const u32x2 e = *(const GLOBAL u32x2*)(vp + (seen ? (int64_t)page * A.page_stride +
                                                                   (int64_t)(at - p * A.page_size) * A.token_stride : 0) * G::ES);
                v[x] = seen ? make_uint2(e.x, e.y) : make_uint2(0, 0);
              }
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const f32x4 e = f32x4{__uint_as_float(v[x].x << 16), __uint_as_float(v[x].x & 0xFFFF0000u),
                                      __uint_as_float(v[x].y << 16), __uint_as_float(v[x].y & 0xFFFF0000u)};
#pragma unroll
                for (int k = 0; k < 4; ++k) sum[k] += isfinite(e[k]) ? 0.f : e[k];
              }
            }
          };
          if constexpr (FORM == ATT_SINKS) {  // (the sinks' tiles, then the others; what is counted twice is not finite twice)
            const int x0 = min(t0, R.sink), x1 = min(t0 + cnt, R.sink), y = R.first - R.sink;
            for (int part = 0; part < 2; ++part) {
              const int a = (part ? max(t0, R.sink) + y : x0) * TILE, b = min(n, (part ? max(t0 + cnt, R.sink) + y : x1) * TILE);
              for (int seen = 0; seen < 2; ++seen) look(seen ? max(a, lo) : a, seen ? b : min(b, A.sinks));
            }
          } else {
            look(max(lo, (R.first + t0) * TILE), min(n, (R.first + t0 + cnt) * TILE));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = sum[k] != 0.f ? sum[k] : o[k];
        }
      }
      if (whole) {
        put(g, d, o, L);
      } else {
        const uint32_t at = slot * SLOT + g * (DP + 4) * 4;
        st_sys4(part, at + d * 4, o);
        if (d == 0) st_sys4(part, at + DP * 4, f32x4{gm, L, 0.f, 0.f});
      }
    }
    if (!whole) {
      // Groups as large as the loads of one trip to memory, which costs about
      // 1.5 us: 1 row of 8192 positions, 16 query heads over one, 64 pieces of
      // 512 x 4 elements: 37 us by groups of 32, 25 by groups of 8, 21 with two
      // elements a thread at once.
      const int n_pieces = (int)all, sets = E < 256 ? 256 / E : 1, trip = 8 * sets;  // (pieces whose loads are in flight)
      const bool two = n_pieces > (E > 256 ? trip : 2 * trip);
      const int fan = n_pieces <= trip * trip ? trip : n_pieces <= 4 * trip * trip ? 2 * trip : 4 * trip;
      const int group0 = two ? (int)(slice - w0) / fan * fan : 0;
      float* jo = &s_o[0][0][0];
      // level 0: the pieces fan .. of one group (only where they are many);
      // level 1: the groups' results, or the pieces
      for (int level = two ? 0 : 1; level < 2; ++level) {
        const int from = level == 0 ? group0 : 0, stride = level == 1 && two ? fan : 1;
        const int np = level == 0 ? min(fan, n_pieces - group0) : (n_pieces + stride - 1) / stride;
        const uint32_t first = from == 0 ? slot0 : 2 * (w0 + from);
        int32_t* count = A.count + ATT_ARRIVALS + (level ? ATT_PLACES * gridDim.x : 0) + first;
        wait_vm_all();
        __syncthreads();
        if (tid == 0) {
          s_last = arrive(count) == np - 1;
          if (s_last) reset_counter(count);
        }
        __syncthreads();
        if (!s_last) break;
        // Y elements a thread at once, so that their loads share one trip to memory
        const auto join = [&](auto at_once) {
          constexpr int Y = at_once;
          for (int e0 = 0; e0 < E; e0 += 256 * Y) {
            const int set = sets > 1 ? tid / E : 0;
            int g[Y], d[Y];
            bool on[Y];
            float gm[Y], L[Y];
            f32x4 o[Y];
#pragma unroll
            for (int y = 0; y < Y; ++y) {
              const int e = sets > 1 ? tid - set * E : e0 + 256 * y + tid;
              on[y] = set < sets && e < E;
              g[y] = on[y] ? e / (D / 4) : 0, d[y] = on[y] ? 4 * (e - g[y] * (D / 4)) : 0;
              gm[y] = -INFINITY, L[y] = 0.f, o[y] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            if (on[0]) {
              for (int x = set; x < np; x += 8 * sets) {  // (eight pieces' loads in flight)
                f32x4 ml[Y][8], po[Y][8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const int p = min(x + i * sets, np - 1);
                  const uint32_t from_p = (p == 0 ? first : 2 * (w0 + from + p * stride)) * SLOT;
#pragma unroll
                  for (int y = 0; y < Y; ++y) {
                    const uint32_t at = from_p + g[y] * (DP + 4) * 4;
                    ml[y][i] = ld_sys4(part, at + DP * 4);
                    po[y][i] = ld_sys4(part, at + d[y] * 4);
                  }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  if (x + i * sets >= np) break;
#pragma unroll
                  for (int y = 0; y < Y; ++y) {
                    const float xm = stride > 1 ? ml[y][i].z : ml[y][i].x, xl = stride > 1 ? ml[y][i].w : ml[y][i].y;
                    const float mn = fmaxf(gm[y], xm), ref = mn == -INFINITY ? 0.f : mn;
                    const float fa = __builtin_amdgcn_exp2f(gm[y] - ref), fb = __builtin_amdgcn_exp2f(xm - ref);
                    o[y] = o[y] * fa + po[y][i] * fb;
                    L[y] = L[y] * fa + xl * fb;
                    gm[y] = mn;
                  }
                }
              }
            }
            if (Y == 1 && sets > 1) {  // the sets' sums in the sets' order
              if (on[0]) {
                *(f32x4*)&jo[4 * tid] = o[0];
                jo[1024 + 2 * tid] = gm[0], jo[1024 + 2 * tid + 1] = L[0];
              }
              __syncthreads();
              if (on[0] && set == 0) {
                for (int x = 1; x < sets; ++x) {
                  const float xm = jo[1024 + 2 * (tid + x * E)], mn = fmaxf(gm[0], xm), ref = mn == -INFINITY ? 0.f : mn;
                  const float fa = __builtin_amdgcn_exp2f(gm[0] - ref), fb = __builtin_amdgcn_exp2f(xm - ref);
                  o[0] = o[0] * fa + *(const f32x4*)&jo[4 * (tid + x * E)] * fb;
                  L[0] = L[0] * fa + jo[1024 + 2 * (tid + x * E) + 1] * fb;
                  gm[0] = mn;
                }
              }
            }
#pragma unroll
            for (int y = 0; y < Y; ++y)
              if (on[y] && set == 0) {
                if (level) {
                  put(g[y], d[y], o[y], L[y]);
                } else {  // (in the group's first place, whose elements only this thread reads, m and l beside its own)
                  const uint32_t at = first * SLOT + g[y] * (DP + 4) * 4;
                  st_sys4(part, at + d[y] * 4, o[y]);
                  if (d[y] == 0) st_sys2(part, at + DP * 4 + 8, __float_as_uint(gm[y]), __float_as_uint(L[y]));
                }
              }
          }
        };
        if (__builtin_expect(E <= 256, 1))
          join(std::integral_constant<int, 1>{});
        else
          join(std::integral_constant<int, 2>{});
      }
    }
    if (even) break;
    if (last_piece && tid == 0) s_next = next;
    __syncthreads();  // (the next piece reuses the LDS)
    u += taken;
    if (u == base + whole_cost * H) base = u, ++row;
    if (last_piece) slice = (uint32_t)uni((int)s_next), asked = true;
  }
  if (tail && tid == 0 && arrive(A.count + ATT_DONE) == (int)workers - 1) {
    reset_counter(A.count + ATT_QUEUE);
    reset_counter(A.count + ATT_DONE);
  }
}

// Two query tiles at once for more than 16 query heads a key head: K and V are
// read and turned once for both (64 rows of up to 4096 positions, 64 heads over
// one: 84 us without, 54 with; 1 row of 700: 18 and 20, the wider pieces' join).
// fp32 heads of more than 128 elements stay at one: the four waves' sums and
// the queries of two would take 166 KB of LDS. bf16 heads of more than 128
// elements take two although the sums of 32 columns fill the registers: 41 are
// spilled where the head has 256 elements and pages hold multiples of 16
// positions, up to 9 otherwise (64 rows of 3000 positions, 24 heads of 256 over
// one: 62 us, 41 are the bytes').
constexpr bool att_widens(int es, int dp) { return es == 2 || dp <= 128; }

template <typename T, int DP, int MODE, int FORM>
void att_launch(const AttArgs& A, int blocks, hipStream_t s) {
  if (A.page_size % 16)
    hipLaunchKernelGGL((k_paged_attention<T, DP, false, false, MODE, FORM>), dim3(blocks), dim3(256), 0, s, A);
  else if (A.head_dim == DP)
    hipLaunchKernelGGL((k_paged_attention<T, DP, true, true, MODE, FORM>), dim3(blocks), dim3(256), 0, s, A);
  else
    hipLaunchKernelGGL((k_paged_attention<T, DP, true, false, MODE, FORM>), dim3(blocks), dim3(256), 0, s, A);
}

template <typename T, int DP, int FORM>
void att_mode(const AttArgs& A, int blocks, hipStream_t s) {
  if constexpr (att_widens(sizeof(T), DP)) {
    if (A.group > 16) return att_launch<T, DP, ATT_WIDE, FORM>(A, blocks, s);
  }
  if (A.req || A.group > 16)
    att_launch<T, DP, ATT_SHARED, FORM>(A, blocks, s);
  else
    att_launch<T, DP, ATT_ONCE, FORM>(A, blocks, s);
}

// one form's launches, for elements of es bytes and heads of up to dp
template <int FORM>
void att_form(const AttArgs& A, int es, int dp, int blocks, hipStream_t s) {
  if (es == 4) {
    if (dp == 64) att_mode<float, 64, FORM>(A, blocks, s);
    else if (dp == 128) att_mode<float, 128, FORM>(A, blocks, s);
    else att_mode<float, 256, FORM>(A, blocks, s);
  } else {
    if (dp == 64) att_mode<uint16_t, 64, FORM>(A, blocks, s);
    else if (dp == 128) att_mode<uint16_t, 128, FORM>(A, blocks, s);
    else att_mode<uint16_t, 256, FORM>(A, blocks, s);
  }
}

}  // namespace scute
