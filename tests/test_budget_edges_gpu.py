"""Chunk attention, weighed rows and eviction at the ends of their ranges: caches
and weights whose offsets pass 32 bits, the most heads, calls of two plans at
once, and captured calls that share one plan's workspace."""
import numpy as np
import pytest
import torch

from paged_mla_speculative_gb300 import binding as mb
from tests import chunk_util as C
from tests import test_weigh_gpu as TW

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


@pytest.mark.parametrize("page", [1, 64])
def test_slots_whose_offsets_pass_32_bits(page):
    """A cache of 4.5 GB (2^31 elements are 3.7 M slots); requests at its end,
    in its middle and at its beginning."""
    d = TW.make([5, 1], [300, 130], 16, page, seed=1)
    slots = 4000000 // 64 * 64
    units = slots // page
    count = d["kv_indices"].numel()
    where = torch.cat((torch.arange(units - count // 2, units), torch.arange(0, count - count // 2))).int().flip(0)
    cache = torch.zeros(slots, 576, dtype=torch.bfloat16, device="cuda")
    old = d["kv_indices"].long()[:, None] * page + torch.arange(page)
    new = where.long()[:, None] * page + torch.arange(page)
    cache[new.flatten().cuda()] = d["cache"][old.flatten()].cuda()
    with mb.Plan(2, 1, 16, page, slots, 300, torch.float32) as plan:
        g = dict(C.to_cuda(d), cache=cache, kv_indices=where.cuda())
        out, lse = C.attn(plan, g)
        TW.weigh(plan, g)
        torch.cuda.synchronize()
        assert plan.get_error() == 0
        C.assert_close(d, out, lse)
        TW.compare(d, g["weights"])
        # Eviction: the rows that stay, moved to pages at the other end.
        refs = torch.zeros(units, dtype=torch.int32, device="cuda")
        refs[where.long().cuda()] = 1
        free = torch.full((units,), -1, dtype=torch.int32, device="cuda")
        free[:10] = torch.arange(units - 20 - count, units - 10 - count, device="cuda").int()
        height = torch.tensor([10], dtype=torch.int32, device="cuda")
        before = cache[new.flatten().cuda()].clone()
        idx, ptr, lens, w = mb.evict_kv(plan, g["weights"], 100, where.cuda(), g["kv_indptr"], g["kv_lens"], cache, refs, free, height,
                                        recent=7)
        torch.cuda.synchronize()
        assert plan.get_error() == 0 and lens.tolist() == [100, 100]
        ptr, starts = ptr.tolist(), d["kv_indptr"].tolist()
        for b, n in enumerate([300, 130]):
            row = g["weights"][b, :n].cpu().double().numpy().copy()
            row[n - 7:] = np.inf
            kept = np.sort(np.argsort(-row, kind="stable")[:100])
            at = (idx[ptr[b]:ptr[b + 1]].long().cpu()[:, None] * page + torch.arange(page)).flatten()[:100]
            assert torch.equal(cache[at.cuda()], before[starts[b] * page:][torch.from_numpy(kept).cuda()])
    del cache


def test_weights_and_layers_whose_offsets_pass_32_bits():
    """Rows of weights 2^31 floats apart; two layers 2^31 elements apart."""
    d = TW.make([3, 2], [200, 150], 8, 64, seed=2)
    pages = d["cache"].shape[0] // 64
    stride = (1 << 31) // 576 // 64 * 64 * 576 + 64 * 576
    layers = torch.zeros(2 * stride, dtype=torch.bfloat16, device="cuda").as_strided((2, pages * 64, 576), (stride, 576, 1))
    layers.copy_(d["cache"].cuda()[None])
    weights = torch.zeros(2 * ((1 << 31) + 64), device="cuda").as_strided((2, 200), ((1 << 31) + 64, 1))
    weights.copy_(d["weights"])
    with C.plan_for(d) as plan:
        g = dict(C.to_cuda(d), weights=weights, cache=layers[1])
        TW.weigh(plan, g)
        torch.cuda.synchronize()
        assert plan.get_error() == 0
        TW.compare(d, weights)
        free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        held = set(d["kv_indices"].tolist())
        rest = [p for p in range(pages) if p not in held]
        free[:len(rest)] = torch.tensor(rest, dtype=torch.int32)
        refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        refs[d["kv_indices"].long().cuda()] = 1
        idx, ptr, lens, w = mb.evict_kv(plan, weights, 70, g["kv_indices"], g["kv_indptr"], g["kv_lens"], layers, refs, free,
                                        torch.tensor([len(rest)], dtype=torch.int32, device="cuda"), sink=3)
        torch.cuda.synchronize()
        assert plan.get_error() == 0
        starts = d["kv_indptr"].tolist()
        for b, n in enumerate([200, 150]):
            row = weights[b, :n].double().cpu().numpy().copy()
            row[:3] = np.inf
            kept = np.sort(np.argsort(-row, kind="stable")[:70])
            slots = d["kv_indices"][starts[b]:starts[b + 1]].long()[torch.from_numpy(kept) // 64] * 64 + torch.from_numpy(kept) % 64
            at = (idx[ptr[b]:ptr[b + 1]].long().cpu()[:, None] * 64 + torch.arange(64)).flatten()[:70]
            for layer in layers:
                assert torch.equal(layer[at.cuda()].cpu(), d["cache"][slots])
            assert torch.equal(w[b, :70].cpu(), weights[b].cpu()[torch.from_numpy(kept)])
    del layers, weights


def test_the_most_heads():
    d = TW.make([1, 2], [70, 300], 4096, 64, seed=3)
    with C.plan_for(d) as plan:
        g = C.to_cuda(d)
        out, lse = C.attn(plan, g)
        TW.weigh(plan, g)
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    C.assert_close(d, out, lse)
    TW.compare(d, g["weights"])


def test_two_plans_on_two_streams_at_once():
    a, b = TW.make([60, 3], [3000, 500], 32, 64, seed=4), TW.make([2] * 6, [900] * 6, 64, 1, seed=5)
    with C.plan_for(a) as pa, C.plan_for(b) as pb:
        ga, gb = C.to_cuda(a), C.to_cuda(b)
        sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        got = []
        for _ in range(6):
            for plan, g, s in ((pa, ga, sa), (pb, gb, sb)):
                with torch.cuda.stream(s):
                    w = g["weights"].clone()
                got.append((g, C.attn(plan, g, stream=s), TW.weigh(plan, dict(g, weights=w), stream=s)))
        torch.cuda.synchronize()
        assert pa.get_error() == 0 and pb.get_error() == 0
    for (g, (out, lse), w), d in zip(got, [a, b] * 6):
        first = got[0] if d is a else got[1]
        assert torch.equal(out, first[1][0]) and torch.equal(lse, first[1][1]) and torch.equal(w, first[2])
    for d, (_, (out, lse), w) in ((a, got[0]), (b, got[1])):
        C.assert_close(d, out, lse)
        TW.compare(d, w)


def test_captured_calls_that_share_a_plan():
    """Graphs of different calls of one plan, replayed in any order in a stream."""
    d, e = TW.make([60, 3], [900, 500], 32, 64, seed=6), TW.make([1, 200], [640, 900], 32, 64, seed=7)
    n = max(d["cache"].shape[0], e["cache"].shape[0])
    for x in (d, e):
        x["cache"] = torch.cat((x["cache"], torch.zeros(n - x["cache"].shape[0], 576).bfloat16()))
    with C.plan_for(d, max_kv_len=900) as plan:
        runs = []
        for x in (d, e):
            g = C.to_cuda(x)
            g["out"], g["l"] = torch.zeros(*g["q"].shape[:2], 512, device="cuda"), torch.zeros(g["q"].shape[:2], device="cuda")
            g["w"] = g["weights"].clone()
            attn, weigh = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
            C.attn(plan, g, out=g["out"], lse=g["l"])
            with torch.cuda.graph(attn):
                C.attn(plan, g, out=g["out"], lse=g["l"])
            with torch.cuda.graph(weigh):
                g["w"].copy_(g["weights"])
                TW.weigh(plan, dict(g, weights=g["w"]))
            runs.append((x, g, attn, weigh))
        for order in ("dDeE", "DdEe", "edDE", "dedDeE"):
            for x, g, _, _ in runs:
                g["out"].zero_(), g["w"].zero_()
            for k in order:
                x, g, attn, weigh = runs[k in "eE"]
                (attn if k.islower() else weigh).replay()
            torch.cuda.synchronize()
            assert plan.get_error() == 0
            for x, g, _, _ in runs:
                C.assert_close(x, g["out"], g["l"])
                TW.compare(x, g["w"])
