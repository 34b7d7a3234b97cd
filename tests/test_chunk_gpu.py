"""Causal attention of chunks of new tokens, through the C ABI, against the
fp64 oracle."""
import numpy as np
import pytest
import torch

from paged_mla_speculative_gb300 import binding as mb
from tests import chunk_util as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def check(d, out_dtype=torch.float32, scale=C.SCALE, **plan_kw):
    with C.plan_for(d, out_dtype, **plan_kw) as plan:
        out, lse = C.attn(plan, C.to_cuda(d), scale)
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    C.assert_close(d, out, lse, scale=scale)


@pytest.mark.parametrize("page", [1, 64])
@pytest.mark.parametrize("new,lens,H", [
    ([1], [1], 1),                                   # one row that sees itself
    ([1], [2], 128),
    ([1], [257], 16),                                # a single token
    ([200], [200], 1),                               # a tile of 128 tokens; nothing cached before
    ([65], [65], 3),                                 # heads that do not divide a tile
    ([130, 1], [130, 300], 20),
    ([7, 0, 3, 0], [128, 40, 260, 0], 16),           # requests without new tokens, one without rows
    ([1] * 9, [1, 64, 65, 127, 128, 129, 256, 257, 700], 64),
    ([300], [1500], 16),
    ([5, 40, 1], [500, 40, 1023], 128),
    ([3], [1000], 200),                              # more heads than a tile has rows
])
def test_matches_the_oracle(new, lens, H, page):
    check(C.make(new, lens, H, page, seed=sum(lens) + H, spike=0.02))


@pytest.mark.parametrize("page", [1, 64])
def test_a_long_context_over_many_clusters(page):
    check(C.make([4], [20000], 32, page, seed=1))    # every tile cut into parts
    check(C.make([40, 1, 1], [9000, 3000, 500], 64, page, seed=2))


def test_more_tiles_than_clusters():
    check(C.make([400], [600], 64, 64, seed=3))
    check(C.make([1] * 100, [130 + 7 * i for i in range(100)], 128, 1, seed=4))


def test_bf16_output_and_scales():
    d = C.make([70, 9], [700, 60], 16, 64, seed=5)
    check(d, torch.bfloat16)
    for scale in (0.5, 1e-3, 0.0, -0.05):
        check(d, scale=scale)


def test_many_requests():
    """Beyond what the layout holds in shared memory."""
    check(C.make([i % 3 for i in range(700)], [i % 3 + i % 41 for i in range(700)], 16, 1, seed=6))


def test_a_plan_without_partials():
    """A plan too small to hold parts of tiles divides the work at their borders."""
    d = C.make([500], [500], 8, 64, seed=7)
    check(d, max_kv_len=512)


def test_tokens_outside_q_indptr_are_left_alone():
    d = C.make([5, 70], [300, 90], 16, 64, seed=8, front=3, pad=9)
    for t in (0, 2, 78, 86):
        d["q"][t] = float("nan")
    g = C.to_cuda(d)
    with C.plan_for(d) as plan:
        out = torch.full((87, 16, 512), 7.0, device="cuda")
        lse = torch.full((87, 16), 7.0, device="cuda")
        C.attn(plan, g, out=out, lse=lse)
        assert plan.get_error() == 0
    outside = [0, 1, 2] + list(range(78, 87))
    assert (out[outside] == 7).all() and (lse[outside] == 7).all()
    C.assert_close(d, out, lse)


def test_equals_the_verify_call_with_a_chain_of_drafts():
    B, T, H = 3, 8, 64
    d = C.make([T] * B, [1000, 300, 77], H, 64, seed=9)
    g = C.to_cuda(d)
    parent = (torch.arange(T, dtype=torch.int32, device="cuda") - 1).repeat(B, 1)
    with C.plan_for(d, T=T) as plan:
        a, la = mb.mla_verify_attn(plan, g["q"].view(B, T, H, 576), g["cache"], g["kv_indices"], g["kv_indptr"], g["kv_lens"], parent,
                                   C.SCALE)
        b, lb = C.attn(plan, g)
        assert plan.get_error() == 0
    C.assert_close(d, b, lb)
    C.assert_close(d, a.view(B * T, H, 512), lb)


@pytest.mark.parametrize("page", [1, 64])
def test_values_that_a_token_does_not_see(page):
    """NaN and infinities in rows behind a request's last (of its page), and in
    rows of later tokens: the tokens before them are not touched."""
    d = C.make([40, 3], [200, 70], 16, page, seed=10)
    slots = {b: s for b, _, _, _, s, _ in C.requests(d)}
    d["cache"][slots[0][180], 100] = float("nan")      # the row of token 20
    d["cache"][slots[0][199], 5] = float("inf")
    if page == 64:
        last = int(slots[0][199])
        d["cache"][last + 1:(last // 64 + 1) * 64] = float("nan")
    d["cache"][slots[1][69], 600 % 576] = 1e6
    with C.plan_for(d) as plan:
        out, lse = C.attn(plan, C.to_cuda(d))
        torch.cuda.synchronize()
        assert plan.get_error() == mb.DEV_RANGE
    assert torch.isnan(out[20:40]).all() and torch.isnan(lse[20:40]).all() and torch.isnan(out[42]).all()
    d["cache"] = torch.nan_to_num(d["cache"].float(), 0, 0, 0).bfloat16()
    C.assert_close(d, out, lse, rows=np.r_[0:20, 40:42])


def test_queries_outside_fp16_touch_their_own_rows_alone():
    d = C.make([30], [300], 16, 64, seed=11)
    d["q"][7, 3, 40] = float("inf")
    d["q"][8, 0, 570] = -1e30
    with C.plan_for(d) as plan:
        out, lse = C.attn(plan, C.to_cuda(d))
        torch.cuda.synchronize()
        assert plan.get_error() == mb.DEV_RANGE
    assert torch.isnan(out[7, 3]).all() and torch.isnan(out[8, 0]).all()
    out[7, 3] = out[8, 0] = 0
    lse[7, 3] = lse[8, 0] = 0
    d["q"][7, 3] = d["q"][8, 0] = 0
    o, l, *_ = C.reference(d)
    out[7, 3], lse[7, 3] = torch.from_numpy(o[7, 3]).cuda(), float(l[7, 3])
    out[8, 0], lse[8, 0] = torch.from_numpy(o[8, 0]).cuda(), float(l[8, 0])
    C.assert_close(d, out, lse)


@pytest.mark.parametrize("page", [1, 64])
def test_bad_slots_are_masked(page):
    d = C.make([2, 5], [3, 200], 16, page, seed=12)
    d["kv_indices"][0] = -1                           # page 64: all of the first request
    if page == 1:
        d["kv_indices"][1:3] = torch.tensor([d["cache"].shape[0], 1 << 30], dtype=torch.int32)
        d["kv_indices"][50] = -7
    else:
        d["kv_indices"][2] = d["cache"].shape[0] // 64
    with C.plan_for(d) as plan:
        out, lse = C.attn(plan, C.to_cuda(d))
        torch.cuda.synchronize()
        assert plan.get_error() == mb.DEV_BAD_SLOT
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all()
    C.assert_close(d, out, lse)


@pytest.mark.parametrize("batch", [4, 600])
def test_requests_that_cannot_be_served_are_nan(batch):
    new, lens = [9, 2, 30, 4] + [1] * (batch - 4), [100, 40, 30, 70] + [3] * (batch - 4)
    d = C.make(new, lens, 16, 64, seed=13, pad=2)
    good = dict(d)
    for name, at, value, bit in (("kv_lens", 1, 1, mb.DEV_BAD_LEN), ("kv_lens", 1, 101, mb.DEV_BAD_LEN),
                                 ("kv_lens", 1, -5, mb.DEV_BAD_LEN), ("kv_indptr", 2, 1, mb.DEV_BAD_INDPTR)):
        d = dict(good)
        d[name] = good[name].clone()
        d[name][at] = value
        with C.plan_for(good) as plan:
            out, lse = torch.full((sum(new) + 2, 16, 512), 7.0).cuda(), torch.full((sum(new) + 2, 16), 7.0).cuda()
            C.attn(plan, C.to_cuda(d), out=out, lse=lse)
            torch.cuda.synchronize()
            assert plan.get_error() == bit
        assert torch.isnan(out[9:11]).all() and torch.isnan(lse[9:11]).all()
        assert (out[sum(new):] == 7).all() and (lse[sum(new):] == 7).all()
        rest = np.r_[0:9, 41:sum(new)] if name == "kv_indptr" else np.r_[0:9, 11:sum(new)]
        C.assert_close(good, out, lse, rows=rest)


@pytest.mark.parametrize("tokens", [[0, 9, 8, 41, 45], [-1, 9, 11, 41, 45], [0, 9, 11, 41, 48]])
def test_tokens_that_are_not_divided_are_all_nan(tokens):
    d = C.make([9, 2, 30, 4], [100, 40, 30, 70], 16, 1, seed=14)
    with C.plan_for(d) as plan:
        g = C.to_cuda(d)
        g["q_indptr"] = torch.tensor(tokens, dtype=torch.int32, device="cuda")
        out, lse = C.attn(plan, g)
        torch.cuda.synchronize()
        assert plan.get_error() == mb.DEV_BAD_INDPTR
        assert torch.isnan(out).all() and torch.isnan(lse).all()
        C.assert_close(d, *C.attn(plan, C.to_cuda(d)))


def test_one_plan_serves_calls_of_other_sizes_in_a_row():
    big = C.make([50, 9, 20], [2000, 700, 300], 16, 64, seed=15)
    with C.plan_for(big, max_batch=8) as plan:
        for new, lens in (([1], [70]), ([300], [1900]), ([2, 2, 2], [500, 2, 64]), ([1] * 8, [2000] * 8)):
            d = C.make(new, lens, 16, 64, seed=sum(lens))
            pages = big["cache"].shape[0] // 64
            cache = torch.zeros_like(big["cache"]) if pages >= d["cache"].shape[0] // 64 else None
            if cache is None:
                continue
            cache[:d["cache"].shape[0]] = d["cache"]
            d["cache"] = cache
            out, lse = C.attn(plan, C.to_cuda(d))
            torch.cuda.synchronize()
            assert plan.get_error() == 0
            C.assert_close(d, out, lse)


def test_captured_and_replayed_with_other_data():
    d = C.make([40, 1, 1], [700, 300, 64], 16, 64, seed=16, pad=3)
    e = C.make([1, 38, 3], [64, 600, 400], 16, 64, seed=17, pad=3)
    n = max(d["cache"].shape[0], e["cache"].shape[0])
    for x in (d, e):
        x["cache"] = torch.cat((x["cache"], torch.zeros(n - x["cache"].shape[0], 576).bfloat16()))
        x["kv_indices"] = torch.cat((x["kv_indices"], torch.zeros(40 - x["kv_indices"].numel(), dtype=torch.int32)))
    with C.plan_for(d, max_kv_len=700) as plan:
        g = C.to_cuda(d)
        eager = C.attn(plan, g)
        out, lse = torch.zeros(45, 16, 512, device="cuda"), torch.zeros(45, 16, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            C.attn(plan, g, out=out, lse=lse)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:42], eager[0][:42]) and torch.equal(lse[:42], eager[1][:42])
        for k in ("q", "cache", "kv_indices", "kv_indptr", "kv_lens", "q_indptr"):
            g[k].copy_(e[k])
        graph.replay()
        torch.cuda.synchronize()
        assert plan.get_error() == 0
        C.assert_close(e, out, lse)


def test_on_another_stream():
    d = C.make([40], [700], 16, 64, seed=18)
    g = C.to_cuda(d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with C.plan_for(d) as plan:
        out, lse = C.attn(plan, g, stream=side)
        side.synchronize()
        assert plan.get_error() == 0
    C.assert_close(d, out, lse)


@pytest.mark.parametrize("fault", [mb.FAULT_EVEN_GIVES_UP, mb.FAULT_ODD_GIVES_UP])
@pytest.mark.parametrize("new,lens,H", [([4], [20000], 32), ([1] * 40, [700] * 40, 64), ([300], [1500], 64)])
def test_every_row_of_a_pair_that_gave_up_is_nan(new, lens, H, fault):
    """(Every pair's first segment has two steps or more here.)"""
    d = C.make(new, lens, H, 64, seed=19)
    g = C.to_cuda(d)
    with C.plan_for(d) as plan:
        plan.inject_fault(fault)
        out, lse = C.attn(plan, g)
        torch.cuda.synchronize()
        assert plan.get_error() == mb.DEV_TIMEOUT
        assert torch.isnan(out).all() and torch.isnan(lse).all()
        out, lse = C.attn(plan, g)
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    C.assert_close(d, out, lse)


def test_no_tokens_and_refusals():
    d = C.make([2, 1], [70, 5], 16, 64, seed=20)
    g = C.to_cuda(d)
    with C.plan_for(d) as plan:
        out, lse = C.attn(plan, dict(g, q=g["q"][:0]))
        assert out.shape == (0, 16, 512) and lse.shape == (0, 16)
        for bad in (dict(g, q=g["q"].float()), dict(g, q=g["q"][:, :8]), dict(g, cache=g["cache"][:-64]),
                    dict(g, kv_lens=g["kv_lens"].long()), dict(g, q_indptr=g["q_indptr"][:2]),
                    dict(g, kv_indptr=g["kv_indptr"][:2]), dict(g, q=g["q"].transpose(0, 1)), dict(g, q=g["q"].cpu())):
            with pytest.raises((TypeError, ValueError)):
                C.attn(plan, bad)
        with pytest.raises(mb.MlaVerifyError):
            C.attn(plan, g, scale=float("nan"))
        for kw in (dict(out=torch.empty(3, 16, 512, dtype=torch.bfloat16, device="cuda")), dict(lse=torch.empty(2, 16, device="cuda"))):
            with pytest.raises((TypeError, ValueError)):
                C.attn(plan, g, **kw)
        lib = mb.load_library()
        p = lambda x: x.data_ptr()  # noqa: E731
        args = [p(g["q"]), p(g["cache"]), p(g["kv_indices"]), p(g["kv_indptr"]), p(g["kv_lens"]), p(g["q_indptr"])]
        o, l = torch.zeros(3, 16, 512, device="cuda"), torch.zeros(3, 16, device="cuda")
        assert lib.mla_verify_attn_chunk(plan.handle, 3, 3, *args, 1.0, p(o), p(l), None) == -4
        assert lib.mla_verify_attn_chunk(plan.handle, 0, 3, *args, 1.0, p(o), p(l), None) == -4
        for n in (-1, (1 << 31) // 16, 1 << 62):
            assert lib.mla_verify_attn_chunk(plan.handle, 2, n, *args, 1.0, p(o), p(l), None) == -9
        for i in range(6):
            assert lib.mla_verify_attn_chunk(plan.handle, 2, 3, *(a if k != i else None for k, a in enumerate(args)), 1.0, p(o), p(l),
                                             None) == -1
            assert lib.mla_verify_attn_chunk(plan.handle, 2, 3, *(a if k != i else a + 4 for k, a in enumerate(args)), 1.0, p(o), p(l),
                                             None) == -2
        assert lib.mla_verify_attn_chunk(None, 2, 3, *args, 1.0, p(o), p(l), None) == -1
        torch.cuda.synchronize()
        assert plan.get_error() == 0
