"""The two-buffer copy of a fork on the host: the order of its steps, and what
it does with a copy that is late or never lands."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_mla_speculative_gb300", "csrc")

# Copies land `delay` ticks after their load (a tick per question or look at
# the clock); prints a line per step, and at the end the time and the copies
# still under way.
HARNESS = r"""
#include "copy_ring.h"
#include <cstdio>
#include <cstdlib>
#include <vector>
struct Ops {
  std::vector<long long> delay, due;
  long long t = 0;
  void load(int i) { due[i] = t + delay[i]; std::printf("load %d\n", i); }
  bool landed(int i) { return due[i] >= 0 && ++t >= due[i]; }
  void store(int i) { std::printf("store %d\n", i); }
  void drain() { std::printf("drain\n"); }
  long long now() { return ++t; }
  void late() { std::printf("late\n"); }
};
int main(int argc, char** argv) {
  Ops o;
  for (int i = 2; i < argc; ++i) o.delay.push_back(std::atoll(argv[i]));
  o.due.assign(o.delay.size(), -1);
  mlav::copy_through_two(o, static_cast<int>(o.delay.size()), std::atoll(argv[1]));
  int under_way = 0;
  for (long long d : o.due) under_way += d > o.t;
  std::printf("end %lld %d\n", o.t, under_way);
}
"""


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cpp").write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(d / "ring.cpp"), "-o", str(d / "ring")], check=True)

    def run(limit, *delays):
        lines = subprocess.run([str(d / "ring"), str(limit), *map(str, delays)], check=True, capture_output=True,
                               text=True).stdout.splitlines()
        end = lines.pop().split()
        return lines, int(end[1]), int(end[2])
    return run


def test_pieces_in_time(ring):
    assert ring(100, 5)[0] == ["load 0", "store 0"]
    lines, _, under_way = ring(100, 5, 50, 1, 1)
    assert lines == ["load 0", "load 1", "store 0", "drain", "load 2", "store 1", "drain", "load 3", "store 2", "store 3"]
    assert under_way == 0


def test_a_late_piece_is_reported_and_used(ring):
    lines, _, under_way = ring(100, 150, 5, 150, 1)
    assert [x for x in lines if x.startswith("store")] == [f"store {i}" for i in range(4)]
    assert lines.count("late") == 2 and under_way == 0


@pytest.mark.parametrize("behind", [1, 250, 290])
def test_the_piece_behind_a_lost_one_lands_before_the_run_ends(ring, behind):
    lines, end, under_way = ring(100, 5, 10 ** 9, behind, 1)
    assert lines[-1] == "late" and "store 0" in lines and "store 1" not in lines and "load 3" not in lines
    assert under_way == 1 and end < 400              # the lost one alone


def test_every_wait_ends(ring):
    lines, end, _ = ring(100, 10 ** 9, 10 ** 9)
    assert lines == ["load 0", "load 1", "late"] and 300 <= end < 320
    lines, end, _ = ring(100, 10 ** 9)
    assert lines == ["load 0", "late"] and 200 <= end < 220
