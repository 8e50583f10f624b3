"""How ragged batches of draft trees are cut into units (csrc/tree_schedule.cuh),
on the CPU: the header's arithmetic, compiled for the host with one lane, over
random batches.  Every (sequence, row block, tile) lies in exactly one unit, no
partial lies past the workspace, and the units fill the CTAs within a stated
bound."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>
#include "tree_schedule.cuh"
using namespace lca;
struct One {
  int lane() const { return 0; }
  int count() const { return 1; }
  int64_t sum(int64_t v) const { return v; }
  template <class I> I scan(I v) const { return v; }
  int first(bool p) const { return p ? 0 : -1; }
  int get(int v, int) const { return v; }
  int64_t get(int64_t v, int) const { return v; }
};
// tree_least_few's search, its 32 lanes one after another
static int least_few(const std::vector<TreeWork>& ws, int most, int64_t limit) {
  int lo = 1, hi = most + 1;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    int at = -1;
    for (int l = 0; l < 32 && at < 0; ++l) {
      const int S = lo + l * step < hi ? lo + l * step : hi;
      int64_t units = 0;
      for (const auto& w : ws) units += (int64_t)w.rb * (S <= most ? (w.tiles + S - 1) / S : 1);
      if (S >= hi || units <= limit) at = l;
    }
    if (at < 0) {
      lo += 31 * step + 1;
    } else {
      const int found = lo + at * step < hi ? lo + at * step : hi;
      lo = at == 0 ? found : lo + (at - 1) * step + 1;
      hi = found;
    }
  }
  return lo;
}
int main() {
  std::mt19937 rng(7);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (int round = 0; round < 400; ++round) {
    const int B = pick(1, round % 7 == 0 ? 700 : 40), G = round % 5 == 0 ? pick(1, 20) : 148;
    const int N = round % 3 == 0 ? 16 : round % 3 == 1 ? 32 : 64, H = pick(1, 128), T = pick(1, 64);
    const int span = 1 << pick(0, 17);
    std::vector<TreeWork> ws(B);
    int most = 1;
    for (auto& w : ws) {
      w = tree_work(pick(0, span), pick(0, T), H, N);
      most = std::max(most, w.tiles);
    }
    auto seq = [&](int b) { return ws[b]; };
    const One one;
    int S = most;
    int64_t best = INT64_MAX;
    for (int k = 1; k <= kTreeMaxWaves; ++k) {
      const int s = tree_least(one, seq, B, most, (int64_t)k * G);
      if (s > 1 && s <= most && tree_units(one, seq, B, s - 1) <= (int64_t)k * G) return printf("not the least\n"), 1;
      const int64_t c = tree_cost(k, s, most);
      if (c < best) best = c, S = s;
      if (B <= 32 && least_few(ws, most, (int64_t)k * G) != s) return printf("the searches differ\n"), 1;
      if (B == 1 && tree_least_few(one, ws[0], B, most, (int64_t)k * G) != s) return printf("the searches differ\n"), 1;
    }
    std::vector<std::vector<int>> seen(B);
    for (int b = 0; b < B; ++b) seen[b].assign((size_t)ws[b].rb * ws[b].tiles, 0);
    const int64_t units = tree_units(one, seq, B, S);
    for (int64_t u = 0; u < units; ++u) {
      const TreeUnit x = u % 2 ? tree_unit<int64_t>(one, seq, B, S, u) : tree_unit<int>(one, seq, B, S, (int)u);
      if (x.b < 0 || x.t0 >= x.t1 || x.t1 - x.t0 > S || x.rb >= ws[x.b].rb || x.part >= x.parts)
        return printf("unit %lld is none\n", (long long)u), 1;
      if (x.parts > 1 && u >= (int64_t)kTreeMaxWaves * G) return printf("a slot past the workspace\n"), 1;
      for (int t = x.t0; t < x.t1; ++t) ++seen[x.b][(size_t)x.rb * ws[x.b].tiles + t];
    }
    if (tree_unit<int64_t>(one, seq, B, S, units).b != -1) return printf("a unit too many\n"), 1;
    for (auto& v : seen)
      for (int c : v)
        if (c != 1) return printf("a tile in %d units\n", c), 1;
    if (best != INT64_MAX && units > (int64_t)kTreeMaxWaves * G) return printf("too many units\n"), 1;
  }
  printf("ok\n");
  return 0;
}
"""


def test_units_cover_every_tile_once(tmp_path):
    src = tmp_path / "schedule.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "schedule"
    subprocess.run(["g++", "-O1", "-std=c++17", "-I" + os.path.join(ROOT, "kv_compression_b200", "csrc"), "-o", str(exe),
                    str(src)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout == "ok\n"


def test_a_cursor_finds_the_same_units(tmp_path):
    """The search that goes on from the last unit found, at the strides of a CTA's units."""
    check = r"""
    for (int64_t c = 0; c < G && c < units; ++c) {
      TreeCursor<int> at;
      for (int64_t u = c; u < units + G; u += G) {
        const TreeUnit x = tree_unit<int>(one, seq, B, S, (int)u, at), y = tree_unit<int>(one, seq, B, S, (int)u);
        if (x.b != y.b || (x.b >= 0 && (x.rb != y.rb || x.part != y.part || x.parts != y.parts || x.t0 != y.t0 || x.t1 != y.t1)))
          return printf("unit %lld differs\n", (long long)u), 1;
        if ((x.b < 0) != (u >= units)) return printf("unit %lld is there or not\n", (long long)u), 1;
      }
    }
    for (auto& v : seen)"""
    at = "\n    for (auto& v : seen)"
    assert at in PROGRAM
    src = tmp_path / "schedule.cpp"
    src.write_text(PROGRAM.replace(at, check, 1).replace("round < 400", "round < 60"))
    exe = tmp_path / "schedule"
    subprocess.run(["g++", "-O1", "-std=c++17", "-I" + os.path.join(ROOT, "kv_compression_b200", "csrc"), "-o", str(exe),
                    str(src)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout == "ok\n"
