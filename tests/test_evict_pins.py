"""Pins of the eviction oracle: small cases by hand, and what must hold of any."""
import math
import random
from types import SimpleNamespace

import pytest
import torch

from oracle import evict_ref as E
from paged_mla_speculative_gb300 import binding


def test_rows_by_hand():
    w = [5.0, 1.0, 3.0, 3.0, 2.0, 3.0, 0.0, 9.0]
    assert E.keep(w, 8, 8, 0, 0) == list(range(8))
    assert E.keep(w, 8, 3, 0, 0) == [0, 2, 7]                      # of the threes, the lowest index
    assert E.keep(w, 8, 4, 0, 0) == [0, 2, 3, 7]
    assert E.keep(w, 8, 4, 2, 1) == [0, 1, 2, 7]                   # protected rows first
    assert E.keep(w, 8, 4, 1, 3) == [0, 5, 6, 7]
    assert E.keep(w, 8, 0, 0, 0) == []
    assert E.keep([0.0, -0.0, 0.0, -1.0], 4, 2, 0, 0) == [0, 1]
    assert E.keep([math.nan, -math.inf, math.nan, math.inf], 4, 3, 0, 0) == [0, 1, 3]


def test_pages_by_hand():
    """A request of three pages cut to 66 rows behind one protected page."""
    n, budget = 192, 66
    w = [0.0] * 192
    w[100], w[150] = 2.0, 1.0
    rows = [[1000 * p + r for p in range(8) for r in range(64)]]
    tables, lens, got, refs, stack, flags = E.evict_kv(
        [w], budget, 64, 0, 3, 64, [4, 2, 6], [0, 3], [n], rows, [0, 0, 2, 0, 1, 0, 1, 0], [0, 1, 7], 8, 256)
    assert flags == 0 and tables == [[4, 7]] and lens == [69] and stack == [0, 1, 6]
    assert refs == [0, 0, 1, 0, 1, 0, 0, 1]                        # page 2 is another table's, too
    assert rows[0][7 * 64:7 * 64 + 3] == [2036, 6022, 7002] and got[0][64:67] == [2.0, 1.0, 0.0]


def test_slots_by_hand():
    tables, lens, got, refs, stack, flags = E.evict_kv(
        [[1.0, 3.0, 2.0, 4.0]], 2, 0, 0, 1, 1, [5, 3, 1, 0, 2], [0, 5], [4], None, [1, 1, 1, 1, 0, 1], [4], 9, 8)
    assert flags == 0 and tables == [[3, 0, 4]] and lens == [3] and got == [[3.0, 4.0, 0.0, 0.0]]
    assert refs == [1, 0, 0, 1, 1, 0] and stack == [1, 2, 5]       # slot 2 was behind the four rows


@pytest.mark.parametrize("page", [1, 64])
def test_what_holds_of_any_case(page):
    rng = random.Random(page)
    for _ in range(60):
        lens = [rng.randint(0, 200) for _ in range(rng.randint(1, 4))]
        budget = rng.randint(0, 220)
        sink = rng.randint(0, budget)
        recent = rng.randint(0, budget - sink)
        extra = rng.choice((0, 1, 70))
        units = 40 if page == 64 else 1500
        ids = list(range(units))
        rng.shuffle(ids)
        tables, ptr = [], [0]
        for n in lens:
            tables.append([ids.pop() for _ in range(-(-n // page))])
            ptr.append(ptr[-1] + len(tables[-1]))
        refs = [0] * units
        for t in tables:
            for u in t:
                refs[u] = 1
        weights = [[rng.choice((0.0, 1.0, rng.random())) for _ in range(300)] for _ in lens]
        rows = [[float(i) for i in range(units * 64)]] if page == 64 else None
        old = list(rows[0]) if rows else None
        new, nl, nw, nrefs, stack, flags = E.evict_kv(weights, budget, sink, recent, extra, page, sum(tables, []), ptr, lens, rows, refs,
                                                      list(ids), 5000, 300)
        assert flags == 0
        held = sum(new, [])
        assert len(set(held)) == len(held) and sorted(held + stack) == list(range(units))    # every unit is held or free
        assert all(nrefs[u] == (1 if u in held else 0) for u in range(units))
        for b, n in enumerate(lens):
            kept = E.keep(weights[b], n, budget, sink, recent)
            assert len(kept) == min(n, budget) and kept == sorted(set(kept)) and nl[b] == len(kept) + extra
            assert len(new[b]) == -(-nl[b] // page)
            if n > budget:
                assert kept[:sink] == list(range(sink)) and kept[len(kept) - recent:] == list(range(n - recent, n))
                free = [j for j in kept if sink <= j < n - recent]
                lost = [j for j in range(sink, n - recent) if j not in free]
                assert not free or not lost or min((weights[b][j], -j) for j in free) > max((weights[b][j], -j) for j in lost)
            at = lambda table, j: table[j // page] * page + j % page  # noqa: E731
            if page == 64:
                assert [rows[0][at(new[b], i)] for i in range(len(kept))] == [old[at(tables[b], j)] for j in kept]
            else:
                assert new[b][:len(kept)] == [tables[b][j] for j in kept]


@pytest.mark.parametrize("size", [5 - 2**32, -2**31 - 1, 2**31, 2**32 + 5])
@pytest.mark.parametrize("name", ["budget", "sink", "recent", "extra_rows"])
def test_sizes_outside_int32_are_refused(name, size):
    """They would reach the library cut off to 32 bits, as other sizes."""
    plan = SimpleNamespace(torch_device=torch.device("cpu"))
    sizes = dict(budget=8, sink=0, recent=0, extra_rows=0) | {name: size}
    with pytest.raises(ValueError, match="32 bits"):
        binding.evict_kv(plan, None, sizes.pop("budget"), None, None, torch.zeros(1, dtype=torch.int32), None, None, None, None,
                         **sizes)


def test_a_cache_without_layers_is_refused():
    plan = SimpleNamespace(torch_device=torch.device("cpu"), num_slots=64)
    with pytest.raises(ValueError, match="layer"):
        binding._expect_layers(plan, torch.zeros((0, 64, 576), dtype=torch.bfloat16))
