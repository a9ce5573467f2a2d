"""How a call of attention over shared positions is cut (csrc/shared_cut.h), for
cards of any number of units: the header is compiled for the host and walked
through. Everything that is to be done is somebody's, and calls smaller than a
workspace was asked for fit it."""

import os
import shutil
import subprocess

import pytest

from lora_normal_form_amd import build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "shared_cut.h"
using namespace scute;

static long failures = 0, looked = 0;
#define CHECK(x, ...) do { ++looked; if (!(x)) { if (++failures < 20) { printf("%s: ", #x); printf(__VA_ARGS__); printf("\n"); } } } while (0)

// each work-group's kind, as the kernel takes it from its number
static void walk(const ShSizes& z, uint32_t units, uint32_t tiles, const char* what, int cu) {
  const ShCut c = sh_cut(z.blocks, units, tiles, z.gang, z.pw);
#define AT "%s: %d units, %d work-groups, gang %d, %u and %u", what, cu, z.blocks, z.gang, units, tiles
  CHECK(c.dies * c.here == (uint32_t)z.blocks && c.ws + c.wo == c.here && c.ws % z.gang == 0, AT);
  CHECK(units == 0 || (uint64_t)c.n_gangs * c.each_s >= units, AT);
  CHECK(tiles == 0 || c.waves > 0, AT);
  CHECK((uint64_t)c.chunks * c.each_o >= tiles, AT);
  CHECK(c.chunks <= (uint64_t)SH_CHUNKS * SH_WAVES * z.blocks, AT);
  CHECK((uint64_t)c.n_gangs * z.gang <= (uint64_t)z.blocks, AT);
  std::vector<int> member(c.n_gangs * z.gang, 0), wave(c.waves, 0);
  for (uint32_t b = 0; b < (uint32_t)z.blocks; ++b) {
    const uint32_t die = b % c.dies, k = b / c.dies, upto = k * c.ws / c.here, next = (k + 1) * c.ws / c.here;
    if (next > upto) {
      const uint32_t gang = die * (c.ws / z.gang) + upto / z.gang, m = upto % z.gang;
      CHECK(gang < c.n_gangs, AT);
      if (gang < c.n_gangs) ++member[gang * z.gang + m];
    } else {
      for (int w = 0; w < SH_WAVES; ++w) {
        const uint32_t x = SH_WAVES * (die * c.wo + k - upto) + w;
        CHECK(x < c.waves, AT);
        if (x < c.waves) ++wave[x];
      }
    }
  }
  for (int n : member) CHECK(n == 1, AT);
  for (int n : wave) CHECK(n == 1, AT);
}

int main() {
  const int64_t calls[][2] = {{1, 1}, {4, 1}, {7, 3}, {64, 1}, {512, 1}, {512, 64}, {5, 0}, {1000, 2}};
  const uint32_t amounts[] = {0, 1, 3, 4, 50, 1000, 100000, 0x7FFFFFFF};
  for (int cu = 1; cu <= 320; ++cu)
    for (int dp : {64, 128, 256})
      for (int es : {2, 4})
        for (int page : {16, 5})
          for (auto& call : calls) {
            const ShSizes z = sh_sizes(es, dp, 1000, 48, page, 32, 8, true, call[0], call[1], cu);
            if (!sh_can_share(z)) {
              CHECK(cu < 2, "%d units share nothing", cu);
              continue;
            }
            for (uint32_t u : amounts)
              for (uint32_t t : amounts)
                if (cu % 16 == 0 || (u + t) % 3 == 0) walk(z, u, t, page == 16 ? "pages of 16" : "pages of 5", cu);
          }
  // work-groups of a join: at most 2^32 threads in a launch, and enough of them
  for (int64_t pairs = 1; pairs <= (int64_t)1 << 34; pairs = pairs * 3 / 2 + 1)
    for (int dp : {64, 128, 256}) {
      const int64_t b = sh_join_blocks(pairs, dp);
      CHECK(b > 0 && b * 256 < (int64_t)1 << 32, "%ld pairs of %d: %ld work-groups", (long)pairs, dp, (long)b);
    }
  srand(7);
  for (int i = 0; i < 200000; ++i) {
    const int64_t rows = rand() % (i % 3 ? 300 : 5000), groups = rand() % (i % 5 ? 40 : 6000);
    const int kv = 1 + rand() % 9, heads = kv * (1 + rand() % (i % 2 ? 10 : 200)), dp = 64 << rand() % 3, es = 2 + 2 * (rand() % 2);
    const int cu = 1 + rand() % 320;
    const int64_t room = sh_workspace(es, dp, 12345, 48, heads, kv, rows, groups, cu);
    for (int j = 0; j < 5; ++j) {
      const int64_t r = rand() % (rows + 1), g = rand() % (groups + 1);
      const ShSizes z = sh_sizes(es, dp, 12345, 48, j % 2 ? 16 : 5, heads, kv, rand() % 2, r, g, cu);
      CHECK(z.bytes <= room, "%ld rows %ld groups of %ld and %ld, %d / %d heads: %ld > %ld", (long)r, (long)g, (long)rows, (long)groups,
            heads, kv, (long)z.bytes, (long)room);
      CHECK(z.rows >= 12345 && z.rows % 256 == 0 && z.seeds % 256 == 0 && z.own % 16 == 0, "alignment");
    }
  }
  printf("%ld checks, %ld failures\n", looked, failures);
  return failures != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_every_unit_and_tile_is_somebodys(tmp_path):
    src, exe = tmp_path / "cut.cpp", tmp_path / "cut"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", build.CSRC, "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:]
    assert os.path.exists(os.path.join(build.CSRC, "shared_cut.h"))
