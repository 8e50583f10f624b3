"""The hand-offs between the tree kernel's MMA warp and its softmax warps, on the
CPU: every order in which the roles can run is walked through, with the barriers
that csrc/tree_events.cuh names.  A waiter knows a phase by its parity alone, so
no barrier may complete a phase before all who wait for the last one have seen
it; and all roles have to come to their end."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kv_compression_b200", "csrc")

PROGRAM = r"""
#include <cstdint>
#include <cstdio>
#include <set>
#include <vector>
#ifdef ONE_BARRIER
namespace lca {
constexpr int kTreeEventBars = 1;
inline int tree_event_bar(int) { return 0; }
inline uint32_t tree_event_parity(int event) { return (uint32_t)event & 1u; }
}
#else
#include "tree_events.cuh"
#endif
using namespace lca;

constexpr int kWarps = 2;
// The MMA warp's doings in order: an event (answered by P, or not), a wait for all P of an event.
enum Kind { kEvent, kWaitP };
struct Op { Kind kind; int no; };
// The softmax warps': a wait for an event, an answer, a meeting of all of them.
enum Step { kWaitEvent, kAnswer, kMeet };
struct Do { Step step; int no; };

struct Program { std::vector<Op> mma; std::vector<Do> soft; };

// Units of the given numbers of tiles; bit i of `back`: the i-th tile comes back.
static Program program(const std::vector<int>& units, unsigned back) {
  Program p;
  int ev = 0, tile = 0, np = 0, meets = 0;
  for (int tiles : units) {
    p.soft.push_back({kMeet, meets++});
    for (int t = 0; t < tiles; ++t, ++tile) {
      for (int turn = 0; turn < (back >> tile & 1u ? 2 : 1); ++turn) {
        p.mma.push_back({kEvent, ev});
        p.soft.push_back({kWaitEvent, ev++});
        p.mma.push_back({kWaitP, np});
        p.soft.push_back({kAnswer, np++});
      }
    }
    p.mma.push_back({kEvent, ev});                 // O
    p.soft.push_back({kWaitEvent, ev++});
    p.soft.push_back({kMeet, meets++});
    p.soft.push_back({kMeet, meets++});
  }
  return p;
}

struct State {
  int mma, soft[kWarps];
  int bar[2], p[2], meet[2];                       // phases completed; of P and the meeting: arrivals in this phase too
  bool operator<(const State& o) const {
    auto key = [](const State& s) { return std::vector<int>{s.mma, s.soft[0], s.soft[1], s.bar[0], s.bar[1], s.p[0], s.p[1], s.meet[0], s.meet[1]}; };
    return key(*this) < key(o);
  }
};

static bool passes(int completed, uint32_t parity) { return ((uint32_t)completed & 1u) != parity; }

// 0: right; 1: a barrier ran ahead of one who waits; 2: someone waits for good.
static int check(const Program& pr) {
  std::set<State> seen;
  std::vector<State> todo(1, State{});
  int worst = 0;
  while (!todo.empty()) {
    const State s = todo.back();
    todo.pop_back();
    if (!seen.insert(s).second) continue;
    bool moved = false;
    auto go = [&](State n) { moved = true; todo.push_back(n); };
    if (s.mma < (int)pr.mma.size()) {
      const Op op = pr.mma[s.mma];
      State n = s;
      ++n.mma;
      if (op.kind == kEvent) {
        ++n.bar[tree_event_bar(op.no)];
        go(n);
      } else if (passes(s.p[0], op.no & 1)) {
        if (s.p[0] != op.no + 1) return 1;
        go(n);
      }
    }
    for (int w = 0; w < kWarps; ++w) {
      if (s.soft[w] == (int)pr.soft.size()) continue;
      const Do d = pr.soft[s.soft[w]];
      State n = s;
      if (d.step == kWaitEvent) {
        const int b = tree_event_bar(d.no), phase = d.no / kTreeEventBars;
        ++n.soft[w];
        if (s.bar[b] > phase + 1) return 1;                    // its parity comes round: this warp would not notice
        if (passes(s.bar[b], tree_event_parity(d.no))) {
          if (s.bar[b] != phase + 1) return 1;
          go(n);
        }
      } else if (d.step == kAnswer) {
        ++n.soft[w];
        if (++n.p[1] == kWarps) ++n.p[0], n.p[1] = 0;
        go(n);
      } else {
        // the meeting, arrival and wait in one: the last to come lets all go on
        bool all = true;
        for (int v = 0; v < kWarps; ++v) all = all && pr.soft[s.soft[v]].step == kMeet && pr.soft[s.soft[v]].no == d.no;
        if (all && w == 0) {
          for (int v = 0; v < kWarps; ++v) ++n.soft[v];
          go(n);
        }
      }
    }
    bool done = s.mma == (int)pr.mma.size();
    for (int w = 0; w < kWarps; ++w) done = done && s.soft[w] == (int)pr.soft.size();
    if (!moved && !done) worst = 2;
  }
  return worst;
}

int main() {
  int walks = 0;
  for (int a = 1; a <= 2; ++a)
    for (int b = 1; b <= 2; ++b)
      for (int c = 1; c <= 2; ++c)
        for (unsigned back = 0; back < 1u << (a + b + c); ++back, ++walks) {
          const int r = check(program({a, b, c}, back));
          if (r) return printf(r == 1 ? "overrun\n" : "stuck\n"), 0;
        }
  printf("ok %d\n", walks);
  return 0;
}
"""


def _walk(tmp_path, *flags):
    src = tmp_path / "events.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "events"
    subprocess.run(["g++", "-O1", "-std=c++17", *flags, "-I" + CSRC, "-o", str(exe), str(src)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout


def test_no_event_overtakes_a_softmax_warp(tmp_path):
    assert _walk(tmp_path) == "ok 216\n"


def test_the_walk_notices_events_on_one_barrier(tmp_path):
    """O of a unit and S of the next on the same barrier: S may be complete before a warp has seen O."""
    assert _walk(tmp_path, "-DONE_BARRIER") == "overrun\n"


@pytest.mark.parametrize("call", [r"mma_commit\(event\b", r"mbar_arrive\(event\b", r"warp_wait\(event\b"])
def test_the_kernel_takes_its_event_barriers_from_there(call):
    with open(os.path.join(CSRC, "tree_tc_kernel.cuh")) as f:
        text = f.read()
    uses = re.findall(call + r"[^,;)]*", text)
    assert uses and all(re.search(r"event \+ tree_event_bar\(ev", u) for u in uses)
