// How a call of attention over shared positions (attend_shared.hip) is cut over a
// card's work-groups, and what of its workspace it needs: arithmetic on sizes, for
// the kernels and the host.
#pragma once

#include <algorithm>
#include <cstdint>

namespace scute {

constexpr int SH_WAVES = 4;         // waves of a work-group
constexpr int SH_CHUNKS = 9;        // chunks a wave at most (eight, and one more)
constexpr float SH_COST_SHARED = 10.f, SH_COST_OWN = 7.f;  // of a unit and of a tile

// The shares of a call's work-groups, `grid` of them, for `units` units of shared
// positions a gang takes and `tiles` tiles of own positions a wave takes.
struct ShCut {
  uint32_t dies, here;        // dies that work-groups go to in turn, work-groups of each
  uint32_t ws, wo;            // of these for shared positions (whole gangs) and for own ones
  uint32_t n_gangs, waves;    // on all dies
  uint32_t each_s, each_o, chunks;  // units of a gang, tiles of a chunk, chunks
};
constexpr ShCut sh_cut(uint32_t grid, uint32_t units, uint32_t tiles, uint32_t gang, uint32_t pw) {
  const auto least = [](uint32_t a, uint32_t b) { return a < b ? a : b; };
  const auto most = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  ShCut c{};
  const float cs = (float)units * gang * SH_COST_SHARED / pw, co = (float)tiles * SH_COST_OWN;
  // (a die needs a gang's work-groups and one for own positions: a partition of 32
  // units, one work-group a unit, is one die)
  c.dies = grid % 8 == 0 && grid / 8 > gang ? 8 : 1, c.here = grid / c.dies;
  if (units) {
    const uint32_t gangs = (uint32_t)((float)c.here * (cs / (cs + co)) / (float)gang + 0.5f);
    c.ws = least(most(gangs, 1u), (c.here - (tiles ? 1 : 0)) / gang) * gang;
  }
  c.wo = c.here - c.ws;
  c.n_gangs = c.dies * (c.ws / gang), c.waves = c.dies * c.wo * SH_WAVES;
  // (four units at least: fewer pieces to join; four rows behind 1000 positions, one unit: 39 us, four: 34)
  c.each_s = c.n_gangs ? most((units + c.n_gangs - 1) / c.n_gangs, 4u) : 1;
  // own tiles: chunks of an eighth of a wave's share (8 tiles at least), taken from
  // a counter after each wave's first: waves with equal work differ by half in time
  const uint32_t share = tiles ? (tiles + c.waves - 1) / c.waves : 1;
  c.each_o = most(least(share, 8u), (share + 7) / 8);
  c.chunks = (tiles + c.each_o - 1) / c.each_o;
  return c;
}

// Work-groups of 256 threads that join the partial results of `pairs` (row, head)s,
// dp / 4 threads each, in turns where there are more: a launch takes 2^32 threads.
constexpr int64_t SH_JOIN_MOST = 65536;
constexpr int64_t sh_join_blocks(int64_t pairs, int dp) {
  const int64_t all = (pairs + 1024 / dp - 1) / (1024 / dp);
  return all < SH_JOIN_MOST ? all : SH_JOIN_MOST;
}

// What a call of these sizes needs.
struct ShSizes {
  int group, cols, cw, pw, gang, together, q_tiles, own_cols, blocks;
  int64_t tiles;                    // (group, key head, wide tile)s at most
  int64_t rows, seeds, own, bytes;  // places in the workspace, and its bytes
};
// es, dp: bytes of an element, elements that heads are padded to; front: bytes before
// the rows' places; units: the card's
inline ShSizes sh_sizes(int es, int dp, int64_t front, int64_t row_bytes, int page_size, int n_heads, int n_kv, bool runs,
                        int64_t n_rows, int64_t n_groups, int units) {
  const auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  ShSizes z;
  z.group = n_heads / n_kv;
  // waves side by side: as many as the columns of a group of the mean size fill,
  // half of them at least; then as many work-groups as it has tiles, up to 4
  const int64_t mean = n_groups > 0 ? n_rows * z.group / n_groups : 0;
  const int wave_cols = dp * es >= 1024 ? 16 : 32;
  z.cw = SH_WAVES;
  if (page_size % 16 == 0)
    while (z.cw > 2 && z.cw / 2 * wave_cols >= mean) z.cw /= 2;
  z.pw = SH_WAVES / z.cw, z.cols = wave_cols * z.cw;
  z.blocks = dp <= 128 ? 2 * units : units;  // (as many as are resident at once)
  z.gang = mean > 2 * z.cols ? 4 : mean > z.cols ? 2 : 1;
  while (z.gang > 1 && z.gang >= z.blocks) z.gang /= 2;
  z.together = runs && z.group <= 8 ? std::min(4, 16 / z.group) : 1;
  z.q_tiles = (z.group + 15) / 16;
  z.own_cols = z.together > 1 ? z.together * z.group : std::min(16, z.group);
  z.tiles = n_kv * (n_rows * z.group / (z.cols * z.gang) + n_groups);
  z.rows = up(front);
  z.seeds = z.rows + up(n_rows * row_bytes);
  z.own = z.seeds + (z.blocks + z.tiles * z.gang) * SH_WAVES * wave_cols * (dp + 4) * 4;
  z.bytes = z.own + (SH_CHUNKS * SH_WAVES * z.blocks + n_rows * n_kv * z.q_tiles) * z.own_cols * (dp + 4) * 4;
  return z;
}
// whether the card holds a gang and a work-group for own positions
constexpr bool sh_can_share(const ShSizes& z) { return z.blocks > 1; }
// and what calls of up to that many rows and groups need, whose waves may stand in
// other ways: a tile and its gang's and turns' take 4 work-groups' columns at most
inline int64_t sh_workspace(int es, int dp, int64_t front, int64_t row_bytes, int n_heads, int n_kv, int64_t max_rows,
                            int64_t max_groups, int units) {
  int64_t bytes = 0;
  for (const bool runs : {false, true}) {
    const ShSizes z = sh_sizes(es, dp, front, row_bytes, 16, n_heads, n_kv, runs, max_rows, max_groups, units);
    const int64_t wave_cols = z.cols / z.cw, all = SH_WAVES * wave_cols;
    const int64_t tiles = (int64_t)n_kv * (max_rows * z.group / (2 * wave_cols) + 4 * max_groups);
    bytes = std::max(bytes, z.bytes + (tiles - z.tiles * z.gang) * all * (dp + 4) * 4);
  }
  return bytes;
}

}  // namespace scute
