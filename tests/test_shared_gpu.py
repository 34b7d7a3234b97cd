"""The verify attention of groups that share their first rows, through the C
ABI, against the fp64 oracle (which knows of no sharing: every request's whole
table), with the tolerances of the verify attention."""
import ctypes
import dataclasses

import numpy as np
import pytest
import torch

from paged_mla_speculative_gb300 import binding as mb
from paged_mla_speculative_gb300 import workloads as W
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def make(sizes, shared, own, T=4, H=16, page_size=1, tree="random", seed=0, spike_frac=0.01, num_slots=None):
    """(inputs on the CPU, group_indptr, shared_lens): group g has sizes[g]
    requests whose first shared[g] rows are one; request b has own[b] more
    rows before its T drafts."""
    group = [g for g, n in enumerate(sizes) for _ in range(n)]
    prefix = tuple(shared[g] + own[b] for b, g in enumerate(group))
    need = sum(-(-(p + T) // 64) * 64 for p in prefix)
    w = W.Workload(name="sh", batch=len(group), num_drafts=T, num_heads=H, prefix=prefix, tree=tree,
                   num_slots=num_slots or -(-need // 1024) * 1024 + 1024, page_size=page_size, spike_frac=spike_frac,
                   seed=seed)
    inp = W.make_inputs(w)
    idx, ptr = inp.kv_indices.clone(), inp.kv_indptr.tolist()
    cache = inp.kv_cache.clone()
    for b, g in enumerate(group):
        first = group.index(g)
        if page_size == 1:
            idx[ptr[b]:ptr[b] + shared[g]] = idx[ptr[first]:ptr[first] + shared[g]]
        else:   # full pages are shared, the rows of a partial one are copies
            full, rest = divmod(shared[g], 64)
            idx[ptr[b]:ptr[b] + full] = idx[ptr[first]:ptr[first] + full]
            if rest:
                a, z = int(idx[ptr[first] + full]) * 64, int(idx[ptr[b] + full]) * 64
                cache[z:z + rest] = cache[a:a + rest]
    gp = torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32)
    return dataclasses.replace(inp, kv_indices=idx, kv_cache=cache), gp, torch.tensor(shared, dtype=torch.int32)


def run(plan, inp, gp, sl, **kw):
    d = G.to_cuda(inp)
    out, lse = mb.mla_verify_attn_shared(plan, d.q, d.kv_cache, d.kv_indices, d.kv_indptr, d.kv_lens, d.draft_parent,
                                         d.scale, gp.cuda(), sl.cuda(), **kw)
    torch.cuda.synchronize()
    return out, lse


def check(case, out_dtype=torch.float32, **plan_kw):
    inp, gp, sl = case
    with G.make_plan(inp, out_dtype, **plan_kw) as plan:
        out, lse = run(plan, inp, gp, sl)
        assert plan.get_error() == 0
    ref_o, ref_l = G.oracle_full(inp)
    if out_dtype == torch.float32:
        return G.assert_parity(out.cpu().numpy(), lse.cpu().numpy(), ref_o, ref_l)
    G.assert_bf16_parity(out.cpu(), lse.cpu().numpy(), ref_o, ref_l)


@pytest.mark.parametrize("page_size", [1, 64])
@pytest.mark.parametrize("sizes,shared,own,T,H", [
    ([1], [0], [0], 1, 1),                                    # one row, its own draft alone
    ([2], [256], [7, 20], 4, 16),                             # two requests in one tile
    ([3], [128], [0, 0, 0], 1, 16),                           # nothing but shared rows and drafts
    ([5], [300], [1, 200, 63, 129, 0], 1, 1),                 # five one-row requests in a tile
    ([2], [130], [500, 3], 8, 64),                            # four tiles a request
    ([9], [1000], [64, 1, 2, 3, 40, 5, 6, 7, 8], 3, 20),      # tiles cut requests at odd rows
    ([2, 3, 1], [512, 64, 200], [10, 20, 30, 0, 400, 5], 4, 16),
    ([0, 2, 0, 1, 0], [77, 256, 0, 0, 9], [10, 20, 30], 2, 16),  # empty groups, a group that shares nothing
])
def test_matches_the_oracle(sizes, shared, own, T, H, page_size):
    check(make(sizes, shared, own, T, H, page_size, seed=sum(shared) + T),
          max_batch=max(len(sizes), sum(sizes)))   # groups are bounded by it as well


@pytest.mark.parametrize("page_size", [1, 64])
def test_long_shared_prefix_over_many_clusters(page_size):
    check(make([2], [20000], [100, 33], 4, 16, page_size, seed=3))
    check(make([3], [9000], [100, 33, 2500], 8, 64, page_size, tree="chain", seed=4))


def test_more_tiles_than_clusters():
    check(make([40], [700], [i % 7 for i in range(40)], 4, 64, seed=5))
    check(make([1] * 90, [130] * 90, [i % 50 for i in range(90)], 1, 128, seed=6))


def test_bf16_output_and_scales():
    case = make([3], [700], [5, 60, 200], 8, 16, seed=7)
    check(case, torch.bfloat16)
    for scale in (0.5, 1e-3):
        check((dataclasses.replace(case[0], scale=scale), *case[1:]))


def test_equals_the_unshared_entry_within_rounding():
    """Groups of one, and a group that shares nothing, are mla_verify_attn."""
    inp, gp, sl = make([4], [0], [300, 2, 1000, 77], 8, 64, seed=8)
    d = G.to_cuda(inp)
    with G.make_plan(inp, max_batch=4) as plan:
        ro, rl = G.run(plan, d)
        one = torch.arange(5, dtype=torch.int32)
        for g, s in ((gp, sl), (one, torch.zeros(4, dtype=torch.int32)), (one, inp.kv_lens - 8)):
            o, l = run(plan, inp, g, s)
            G.assert_parity(o.cpu().numpy(), l.cpu().numpy(), ro.double().cpu().numpy(), rl.double().cpu().numpy())
        assert plan.get_error() == 0


def test_one_plan_serves_calls_of_other_sizes_in_a_row():
    """Every call reads only what it laid out itself: the workspace holds other
    calls' layouts, keys and partials."""
    cases = [make([2, 3, 1], [512, 64, 200], [10, 20, 30, 0, 400, 5], 4, 16, 1, seed=20, num_slots=16384),
             make([1], [5000], [9], 4, 16, 1, seed=21, num_slots=16384),
             make([6], [64], [0, 1, 2, 3, 4, 500], 4, 16, 1, seed=22, num_slots=16384),
             make([1, 1], [100, 1], [0, 3000], 4, 16, 1, seed=23, num_slots=16384)]
    refs = [G.oracle_full(c[0]) for c in cases]
    with mb.Plan(6, 4, 16, 1, 16384, 5200) as plan:
        for k in (0, 1, 2, 3, 0, 2, 1, 3):
            o, l = run(plan, *cases[k])
            G.assert_parity(o.cpu().numpy(), l.cpu().numpy(), *refs[k])
            d = G.to_cuda(cases[k][0])
            o, l = G.run(plan, d)                       # the unshared entry on the same workspace
            G.assert_parity(o.cpu().numpy(), l.cpu().numpy(), *refs[k])
        assert plan.get_error() == 0


def test_more_requests_than_the_shared_memory_layout():
    """600 requests (and groups, and tiles): planned in global memory."""
    n = 600
    inp, gp, sl = make([n], [70], [i % 5 for i in range(n)], 1, 4, seed=9, spike_frac=0.0)
    ref = G.oracle_full(inp)
    with G.make_plan(inp) as plan:
        o, l = run(plan, inp, gp, sl)
        G.assert_parity(o.cpu().numpy(), l.cpu().numpy(), *ref)
        own = torch.arange(n + 1, dtype=torch.int32)    # 600 groups of one
        o, l = run(plan, inp, own, torch.full((n,), 70, dtype=torch.int32))
        G.assert_parity(o.cpu().numpy(), l.cpu().numpy(), *ref)
        assert plan.get_error() == 0


@pytest.mark.parametrize("T,H", [(4, 16), (2, 128)])
def test_bad_requests_are_nan_and_the_others_are_served(T, H):
    inp, gp, sl = make([4, 1], [200, 50], [10, 300, 5, 40, 30], T, H, seed=10)
    ref_o, ref_l = G.oracle_full(inp)

    def expect(inp, gp, sl, bad, flag):
        with G.make_plan(inp, max_kv_len=600) as plan:
            o, l = run(plan, inp, gp, sl)
            assert plan.get_error() == flag
        for b in range(5):
            if b in bad:
                assert torch.isnan(o[b]).all() and torch.isnan(l[b]).all()
            else:
                G.assert_parity(o[b].cpu().numpy(), l[b].cpu().numpy(), ref_o[b], ref_l[b])
    lens = inp.kv_lens.clone()
    lens[1] = T - 1
    expect(dataclasses.replace(inp, kv_lens=lens), gp, sl, [1], mb.DEV_BAD_LEN)
    lens[1] = 601
    expect(dataclasses.replace(inp, kv_lens=lens), gp, sl, [1], mb.DEV_BAD_LEN)
    lens = inp.kv_lens.clone()
    lens[0] += 1                                         # the group's first request: its table is not read
    expect(dataclasses.replace(inp, kv_lens=lens), gp, sl, [0], mb.DEV_BAD_INDPTR)
    expect(inp, gp, torch.tensor([200, 81], dtype=torch.int32), [4], mb.DEV_BAD_LEN)
    expect(inp, gp, torch.tensor([-1, 50], dtype=torch.int32), [0, 1, 2, 3], mb.DEV_BAD_LEN)
    for groups in ([0, 4, 4], [1, 4, 5], [0, 6, 5], [0, -1, 5]):
        expect(inp, torch.tensor(groups, dtype=torch.int32), sl, range(5), mb.DEV_BAD_INDPTR)


def test_bad_slots_and_parents():
    T = 4
    inp, gp, sl = make([3], [200], [10, 300, 5], T, 16, seed=11)
    idx, ptr = inp.kv_indices.clone(), inp.kv_indptr.tolist()
    idx[7] = inp.kv_cache.shape[0]                       # a shared key, through the first request's table
    idx[ptr[1] + 250] = -3                               # an own key of the second request
    with G.make_plan(inp) as plan:
        o, l = run(plan, dataclasses.replace(inp, kv_indices=idx), gp, sl)
        assert plan.get_error() == mb.DEV_BAD_SLOT
    keep = torch.ones(len(idx), dtype=torch.bool)
    for b in range(3):
        keep[ptr[b] + 7] = False
    keep[ptr[1] + 250] = False
    lens = inp.kv_lens - torch.tensor([1, 2, 1], dtype=torch.int32)
    ref = dataclasses.replace(inp, kv_indices=inp.kv_indices[keep], kv_lens=lens,
                              kv_indptr=torch.cat((torch.zeros(1, dtype=torch.int32), lens.cumsum(0).int())))
    G.assert_parity(o.cpu().numpy(), l.cpu().numpy(), *G.oracle_full(ref))
    par = inp.draft_parent.clone()
    par[1, 2] = 3
    want = inp.draft_parent.clone()
    want[1, 2] = -1
    with G.make_plan(inp) as plan:
        o, l = run(plan, dataclasses.replace(inp, draft_parent=par), gp, sl)
        assert plan.get_error() == mb.DEV_BAD_PARENT
    G.assert_parity(o.cpu().numpy(), l.cpu().numpy(), *G.oracle_full(dataclasses.replace(inp, draft_parent=want)))


def test_every_key_of_a_row_masked():
    """A request whose whole table lies outside the cache: weight 0, lse -inf."""
    inp, gp, sl = make([1, 1], [0, 0], [300, 5], 2, 16, seed=12)
    idx = inp.kv_indices.clone()
    idx[:302] = -1
    with G.make_plan(inp) as plan:
        o, l = run(plan, dataclasses.replace(inp, kv_indices=idx), gp, sl)
        assert plan.get_error() == mb.DEV_BAD_SLOT
    assert (o[0] == 0).all() and (l[0] == -np.inf).all()
    ro, rl = G.oracle_full(inp)
    G.assert_parity(o[1].cpu().numpy(), l[1].cpu().numpy(), ro[1], rl[1])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e30])
def test_values_outside_fp16_reach_only_the_rows_that_see_them(value):
    T = 4
    inp, gp, sl = make([3, 1], [200, 100], [10, 300, 5, 20], T, 16, tree="star", seed=13)
    ro, rl = G.oracle_full(inp)
    ptr = inp.kv_indptr.tolist()
    P = (inp.kv_lens - T).tolist()

    def with_bad(b, j, dim):
        cache = inp.kv_cache.clone()
        cache[int(inp.kv_indices[ptr[b] + j]), dim] = value
        with G.make_plan(inp) as plan:
            o, l = run(plan, dataclasses.replace(inp, kv_cache=cache), gp, sl)
            assert plan.get_error() == mb.DEV_RANGE
        return o, l

    def rows(o, l, lost):
        for b in range(4):
            for t in range(T):
                if (b, t) in lost:
                    assert torch.isnan(o[b, t]).all() and torch.isnan(l[b, t]).all(), (b, t)
                else:
                    G.assert_parity(o[b, t].cpu().numpy(), l[b, t].cpu().numpy(), ro[b, t], rl[b, t])
    every = lambda *bs: [(b, t) for b in bs for t in range(T)]  # noqa: E731
    rows(*with_bad(0, 150, 3), every(0, 1, 2))             # a shared row: its group
    rows(*with_bad(1, 250, 511), every(1))                 # an own row: its request, in tiles with others
    rows(*with_bad(2, P[2] + 1, 575), [(2, 1)])            # a draft nobody else sees
    q = inp.q.clone()
    q[1, 2, 5, 17] = value
    with G.make_plan(inp) as plan:
        o, l = run(plan, dataclasses.replace(inp, q=q), gp, sl)
        assert plan.get_error() == mb.DEV_RANGE
    o, l = o.clone(), l.clone()
    assert not torch.isfinite(o[1, 2, 5]).all()
    o[1, 2, 5], l[1, 2, 5] = torch.from_numpy(ro[1, 2, 5]).to(o), float(rl[1, 2, 5])
    G.assert_parity(o.cpu().numpy(), l.cpu().numpy(), ro, rl)


def test_rows_behind_the_batch_stay_as_they_were():
    inp, gp, sl = make([2], [130], [40, 7], 3, 20, seed=14)
    d = G.to_cuda(inp)
    out = torch.full((4, 3, 20, 512), 7.0, device="cuda")
    lse = torch.full((4, 3, 20), 7.0, device="cuda")
    with G.make_plan(inp, max_batch=5) as plan:
        mb.mla_verify_attn_shared(plan, d.q, d.kv_cache, d.kv_indices, d.kv_indptr, d.kv_lens, d.draft_parent, d.scale, gp.cuda(),
                                  sl.cuda(), out[:2], lse[:2])
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    assert (out[2:] == 7).all() and (lse[2:] == 7).all()
    G.assert_parity(out[:2].cpu().numpy(), lse[:2].cpu().numpy(), *G.oracle_full(inp))


def test_rows_beyond_the_32_bit_offset():
    """The same requests in the last rows of a cache of 2.4e9 elements."""
    inp, gp, sl = make([3], [700], [30, 200, 5], 4, 16, seed=51)
    ref = G.oracle_full(inp)
    n, small = (1 << 22) + 64, inp.kv_cache.shape[0]
    cache = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda")
    cache[n - small:] = inp.kv_cache.cuda()
    moved = dataclasses.replace(inp, kv_cache=cache, kv_indices=inp.kv_indices + (n - small))
    with G.make_plan(moved) as plan:
        o, l = run(plan, moved, gp, sl)
        assert plan.get_error() == 0
    G.assert_parity(o.cpu().numpy(), l.cpu().numpy(), *ref)


def test_longest_trees_and_most_heads():
    """32 drafts (every ancestor bit), 4096 query rows a request."""
    check(make([2], [300], [40, 7], 32, 128, seed=52))


def test_captured_and_replayed_with_other_lengths_and_groups():
    T, H = 4, 64
    cases = [make([3, 1], [300, 100], [10, 20, 30, 40], T, H, 64, seed=31, num_slots=8192),
             make([1, 3], [64, 900], [700, 2, 3, 4], T, H, 64, seed=32, num_slots=8192),
             make([4, 0], [0, 0], [1, 1000, 3, 600], T, H, 64, seed=33, num_slots=8192)]
    most = max(c[0].kv_indices.numel() for c in cases)
    dev = "cuda"
    first = cases[0][0]
    buf = dict(q=torch.empty_like(first.q, device=dev), kv_cache=torch.empty_like(first.kv_cache, device=dev),
               kv_indices=torch.zeros(most, dtype=torch.int32, device=dev),
               kv_indptr=torch.zeros(5, dtype=torch.int32, device=dev), kv_lens=torch.zeros(4, dtype=torch.int32, device=dev),
               draft_parent=torch.zeros((4, T), dtype=torch.int32, device=dev))
    g_, s_ = torch.zeros(3, dtype=torch.int32, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)

    def load(c):
        for k, v in buf.items():
            src = getattr(c[0], k)
            v.view(-1)[:src.numel()].copy_(src.view(-1))
        g_.copy_(c[1])
        s_.copy_(c[2])
        torch.cuda.synchronize()
    with mb.Plan(4, T, H, 64, 8192, 1100) as plan, mb.Plan(4, T, H, 64, 8192, 1100) as other:
        out, lse = plan.new_outputs(4)
        s = torch.cuda.Stream()
        load(cases[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            mb.mla_verify_attn_shared(plan, *buf.values(), first.scale, g_, s_, out, lse, stream=s)
        for c in cases + cases[::-1]:
            load(c)
            g.replay()
            torch.cuda.synchronize()
            o, l = mb.mla_verify_attn_shared(other, *buf.values(), first.scale, g_, s_)
            torch.cuda.synchronize()
            assert torch.equal(o, out) and torch.equal(l, lse)      # the same bits eagerly, by another plan
            G.assert_parity(out.cpu().numpy(), lse.cpu().numpy(), *G.oracle_full(c[0]))
        assert plan.get_error() == 0 and other.get_error() == 0


def test_two_plans_on_two_streams_at_once():
    cases = [make([5], [3000], [9, 100, 3, 0, 50], 8, 64, seed=41), make([2, 2], [800, 2000], [9, 100, 3, 0], 8, 64, seed=42)]
    ins = [(G.to_cuda(c[0]), c[1].cuda(), c[2].cuda()) for c in cases]
    plans = [G.make_plan(c[0]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for k, (d, g, sl) in enumerate(ins):
            with torch.cuda.stream(streams[k]):
                outs[k].append(mb.mla_verify_attn_shared(plans[k], d.q, d.kv_cache, d.kv_indices, d.kv_indptr, d.kv_lens,
                                                         d.draft_parent, d.scale, g, sl))
    torch.cuda.synchronize()
    for k, c in enumerate(cases):
        ref = G.oracle_full(c[0])
        for o, l in outs[k]:
            assert torch.equal(o, outs[k][0][0]) and torch.equal(l, outs[k][0][1])
        G.assert_parity(outs[k][0][0].cpu().numpy(), outs[k][0][1].cpu().numpy(), *ref)
        assert plans[k].get_error() == 0
        plans[k].close()


def test_host_argument_errors():
    inp, gp, sl = make([2], [100], [1, 2], 4, 16, seed=50)
    d, g, s = G.to_cuda(inp), gp.cuda(), sl.cuda()
    with G.make_plan(inp) as plan:
        lib = mb.load_library()
        out, lse = plan.new_outputs(2)

        def call(batch=2, scale=0.1, groups=1, **over):
            ptr = dict(q=d.q, kv=d.kv_cache, idx=d.kv_indices, indptr=d.kv_indptr, lens=d.kv_lens, par=d.draft_parent, g=g, s=s,
                       out=out, lse=lse)
            x = {k: over[k] if k in over else v.data_ptr() for k, v in ptr.items()}
            return lib.mla_verify_attn_shared(plan.handle, batch, x["q"], x["kv"], x["idx"], x["indptr"], x["lens"], x["par"],
                                              ctypes.c_float(scale), groups, x["g"], x["s"], x["out"], x["lse"], None)
        assert call() == 0
        for k in ("q", "kv", "idx", "indptr", "lens", "par", "g", "s", "out", "lse"):
            assert call(**{k: None}) == -1 and call(**{k: d.q.data_ptr() + 8}) == -2, k
        assert call(batch=0) == -4 and call(batch=3) == -4
        assert call(scale=float("nan")) == -5 and call(scale=float("inf")) == -5
        assert call(groups=0) == -9 and call(groups=3) == -9
        torch.cuda.synchronize()
        assert plan.get_error() == 0
