"""What evict_kv writes lies in nothing else that it is given: the check of
address ranges compiled for the host, against bytes one by one, and the
binding's check of the table, which the library knows the beginning of alone."""
import os
import random
import shutil
import subprocess
import types

import pytest
import torch

from paged_mla_speculative_gb300 import binding as mb

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_mla_speculative_gb300", "csrc")

HARNESS = r"""
#include "spans.h"
#include <cstdio>
int main() {
  long long a[4], b[4];
  while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld", a, a + 1, a + 2, a + 3, b, b + 1, b + 2, b + 3) == 8) {
    const mlav::Span x = mlav::row_span(reinterpret_cast<void*>(a[0]), a[1], a[2], a[3]);
    const mlav::Span y = mlav::row_span(reinterpret_cast<void*>(b[0]), b[1], b[2], b[3]);
    const mlav::Span z = mlav::flat_span(reinterpret_cast<void*>(1LL << 40), 5);
    const mlav::Span both[2] = {x, z};
    const bool o = mlav::overlap(x, y);
    const bool same = o == mlav::overlap(y, x) && o == mlav::any_overlap(both, 2, &y, 1) && !mlav::any_overlap(both, 2, &z, 0);
    std::printf("%d\n", same ? o : 2);
  }
}
"""


def test_overlaps_are_those_of_the_bytes(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    (tmp_path / "spans.cpp").write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(tmp_path / "spans.cpp"), "-o", str(tmp_path / "spans")], check=True)
    rng = random.Random(1)

    def span():
        rows, size = rng.choice((0, 1, 1, 2, 5)), rng.choice((0, 1, 4, 7))
        return rng.randrange(1000, 1060), rows, rng.choice((0,) if rows <= 1 else (size, size + 1, size + 9)) if rows <= 1 or size else 9, size

    def bytes_of(s):
        return {s[0] + i * s[2] + k for i in range(s[1]) for k in range(s[3])}

    cases = [(span(), span()) for _ in range(4000)]
    # Weights and new weights side by side, as [requests, 2, width]; tables between the rows of a strided cache.
    cases += [((1000, 8, 80, 40), (1040, 8, 80, 40)), ((1000, 8, 80, 40), (1039, 8, 80, 40)), ((1000, 3, 100, 60), (1160, 1, 0, 40)),
              ((1000, 3, 100, 60), (1160, 1, 0, 41)), ((1000, 3, 100, 60), (1159, 1, 0, 5))]
    out = subprocess.run([str(tmp_path / "spans")], input="\n".join(" ".join(map(str, a + b)) for a, b in cases), capture_output=True,
                         text=True, check=True).stdout.split()
    want = ["1" if bytes_of(a) & bytes_of(b) else "0" for a, b in cases]
    assert out == want and "1" in want and "0" in want


class Library:
    """Takes calls in the place of the library."""

    def __init__(self):
        self.calls = 0

    def mla_verify_evict_kv(self, *args):
        self.calls += 1
        return 0


def test_the_binding_refuses_outputs_in_the_table(monkeypatch):
    lib = Library()
    monkeypatch.setattr(mb, "load_library", lambda path=None: lib)
    monkeypatch.setattr(mb, "strerror", lambda status: "refused")
    monkeypatch.setattr(mb, "_stream_ptr", lambda stream: 0)
    plan = types.SimpleNamespace(torch_device=torch.device("cpu"), max_kv_len=100, num_slots=256, page_size=64, handle=0)
    memory = torch.zeros(400, dtype=torch.int32)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    args = dict(weights=torch.zeros(2, 100), budget=64, kv_indices=memory[100:140], kv_indptr=i32(0, 2, 4), kv_lens=i32(100, 100),
                kv_cache=torch.zeros(256, 576, dtype=torch.bfloat16), page_refs=torch.zeros(4, dtype=torch.int32),
                free_pages=torch.zeros(4, dtype=torch.int32), free_count=i32(0), new_indices=torch.zeros(8, dtype=torch.int32),
                new_indptr=i32(0, 0, 0), new_lens=i32(0, 0), new_weights=torch.zeros(2, 100))
    for inside in (dict(new_indices=memory[90:101]), dict(new_indices=memory[136:150]), dict(new_indptr=memory[120:123]),
                   dict(new_lens=memory[138:140]), dict(page_refs=memory[97:101]), dict(free_pages=memory[104:108]),
                   dict(free_count=memory[139:140]), dict(new_indices=memory)):
        with pytest.raises(mb.MlaVerifyError):
            mb.evict_kv(plan, **dict(args, **inside))
    assert lib.calls == 0
    for beside in ({}, dict(new_indices=memory[80:100]), dict(new_indices=memory[140:160]), dict(new_lens=memory[140:142])):
        mb.evict_kv(plan, **dict(args, **beside))
    assert lib.calls == 4
