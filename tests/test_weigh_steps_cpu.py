"""The closed form of the steps of weighed rows against sums of the
definition, compiled for the host."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_mla_speculative_gb300", "csrc")

HARNESS = r"""
#include "weigh_steps.h"
#include <cstdio>
int main() {
  long long n, c, H;
  while (std::scanf("%lld %lld %lld", &n, &c, &H) == 3) {
    mlav::WeighSteps s(n, c, H);
    long long sum = 0;
    const long long tiles = (c * H + 255) / 256, blocks = c ? (n + 255) / 256 : 0;
    bool ok = s.tiles == tiles && s.blocks == blocks && s.before(0) == 0;
    const long long near = blocks < 3000 ? 0 : blocks - 3000;   // (long ones: the end alone)
    if (near) sum = s.before(near);
    for (long long kb = near; kb < blocks; ++kb) {
      // the first tile that holds a row of a token that sees the block's first key
      const long long token = 256 * kb > n - c ? 256 * kb - (n - c) : 0, first = token * H / 256;
      ok = ok && s.first(kb) == first && first < tiles && s.block_at(sum) == kb && s.block_at(sum + tiles - first - 1) == kb;
      sum += tiles - first;
      ok = ok && s.before(kb + 1) == sum;
    }
    if (near && c == 1) ok = ok && s.before(near) == near * tiles;
    ok = ok && s.total() == sum;
    std::printf("%d\n", ok ? 1 : 0);
  }
}
"""


def test_steps_and_sums(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    (tmp_path / "steps.cpp").write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(tmp_path / "steps.cpp"), "-o", str(tmp_path / "steps")], check=True)
    cases = [(n, c, H) for H in (1, 2, 3, 16, 20, 64, 100, 256, 257, 4096) for c in (0, 1, 2, 5, 64, 255, 256, 257, 1001)
             for n in (c, c + 1, c + 255, c + 256, c + 257, c + 5000, 2000000000)]
    out = subprocess.run([str(tmp_path / "steps")], input="\n".join("%d %d %d" % x for x in cases), capture_output=True, text=True,
                         check=True).stdout.split()
    assert len(out) == len(cases)
    assert [x for x, ok in zip(cases, out) if ok != "1"] == []
