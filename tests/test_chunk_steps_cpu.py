"""The closed form of a chunk's tiles and steps against sums of the definition,
compiled for the host."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_mla_speculative_gb300", "csrc")

HARNESS = r"""
#include "chunk_steps.h"
#include <cstdio>
int main() {
  long long n, c, H;
  while (std::scanf("%lld %lld %lld", &n, &c, &H) == 3) {
    mlav::ChunkSteps s(n, c, H, 3, 2);
    long long sum = 0;
    const long long tiles = (c * H + 127) / 128;
    bool ok = s.tiles == tiles && s.before(0) == 0;
    for (long long t = 0; t < tiles; ++t) {
      const long long end = 128 * t + 128 < c * H ? 128 * t + 128 : c * H;   // of its rows
      const long long keys = n - c + (end - 1) / H + 1;
      const long long steps = (keys + 255) / 256;
      ok = ok && s.steps(t) == steps && s.tile_at(sum) == t && s.tile_at(sum + 3 * steps + 1) == t;
      sum += 3 * steps + 2;
      ok = ok && s.before(t + 1) == sum;
    }
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
    cases = [(n, c, H) for H in (1, 2, 3, 16, 20, 64, 100, 128, 129, 200, 4096) for c in (1, 2, 5, 64, 127, 300, 1001)
             for n in (c, c + 1, c + 255, c + 256, c + 257, c + 5000, 2000000000)]
    out = subprocess.run([str(tmp_path / "steps")], input="\n".join("%d %d %d" % x for x in cases), capture_output=True, text=True,
                         check=True).stdout.split()
    assert len(out) == len(cases)
    assert [x for x, ok in zip(cases, out) if ok != "1"] == []
