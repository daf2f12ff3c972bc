"""The turns of the layer norm's rings of copies (csrc/ring.h), compiled for the host and held against a plain account of every copy
asked for: in order, and after a wait that gave up, where exactly the copies under way are waited for, each in its own stage and
phase, and no stage that nothing fills any more."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

MODEL = r"""
#include <cstdio>
#include <set>
#include <utility>
#include "ring.h"
using fxtx::RingTurn;

#define CHECK(x) if (!(x)) { std::printf("stages %d items %d first %d step %d fails at %d: %s\n", stages, items, first, step, fails, #x); return 1; }

// A copying thread takes items first, first + step, ... below `items`; its wait for the `fails`-th of them gives up (-1: none does).
int run(int stages, int items, int first, int step, int fails) {
  RingTurn turn(stages);
  int filled[64] = {};                       // of a stage: fills asked for, each completing the barrier's next phase
  std::set<std::pair<int, int>> under_way;   // (stage, phase) of the copies asked for and not waited for
  auto fill = [&](int stage, int item) {
    if (item >= items) return;
    under_way.insert({stage, filled[stage]++ & 1});
  };
  for (int x = 0; x < stages; ++x) fill(x, first + x * step);
  int at = 0;
  for (int item = first; item < items; item += step, ++at) {
    if (at == fails) {
      for (int x = 0; x < stages; ++x)
        if (turn.asked(x, item, items, step)) CHECK(under_way.erase({x, (int)turn.parity(x)}) == 1);
      CHECK(under_way.empty());
      return 0;
    }
    CHECK(under_way.erase({turn.s, (int)turn.phase}) == 1);
    fill(turn.s, item + stages * step);
    turn.next();
  }
  CHECK(under_way.empty());
  return 0;
}

int main() {
  long n = 0;
  for (int stages = 1; stages <= 8; ++stages)
    for (int items = 0; items <= 40; ++items)
      for (int step : {1, 2, 7})
        for (int first = 0; first < step + 2; ++first)
          for (int fails = -1; fails <= items; ++fails, ++n)
            if (run(stages, items, first, step, fails)) return 1;
  std::printf("%ld\n", n);
  return 0;
}
"""


def test_every_copy_under_way_is_waited_for(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    (tmp_path / "model.cpp").write_text(MODEL)
    csrc = os.path.join(ROOT, "dense_linear_algebra_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-I", csrc, str(tmp_path / "model.cpp"), "-o", str(tmp_path / "model")], check=True)
    got = subprocess.run([str(tmp_path / "model")], capture_output=True, text=True)
    assert got.returncode == 0 and int(got.stdout) > 10_000, got.stdout


def test_the_kernels_take_their_turns_from_there():
    """No ring of norm.cu keeps a stage or a phase of its own, each loop over rows ends at its first wait that gave up, and each
    copying thread then drains."""
    source = open(os.path.join(ROOT, "dense_linear_algebra_gb300", "csrc", "norm.cu")).read()
    assert "phase ^=" not in source and source.count("RingTurn turn") == 3
    assert source.count("if (!ring.wait()) break;") == source.count("  leave_rows<") == 4
    assert source.count("drain(full, turn, tile, tiles, step);") == source.count("drain(ring.full, ring.turn, row, rows, step);") == 1
