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
