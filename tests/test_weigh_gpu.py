"""The attention weight given to cached rows, through the C ABI, against the
fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import chunk_ref, evict_ref
from paged_mla_speculative_gb300 import binding as mb
from tests import chunk_util as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def make(new, lens, H, page=1, seed=0, scale=C.SCALE, extra=0, **kw):
    """chunk_util's inputs with the log-sum-exps of the tokens (by the oracle,
    rounded to fp32) and weights that hold something already."""
    d = C.make(new, lens, H, page, seed, spike=0, **kw)
    N = d["q"].shape[0]
    lse = np.zeros((N, H))
    for b, t0, t1, n, slots, ok in C.requests(d):
        if t1 > t0:
            lse[t0:t1] = chunk_ref.chunk_attn(d["q"][t0:t1].double().numpy(), C.gather(d, slots, ok), scale, ok)[1]
    d["lse"] = torch.from_numpy(lse).float()
    g = torch.Generator().manual_seed(seed + 1)
    d["weights"] = torch.rand(len(lens), max(max(lens), 1) + extra, generator=g)
    return d


def weigh(plan, d, scale=C.SCALE, **kw):
    return mb.weigh_kv(plan, d["q"], d["cache"], d["kv_indices"], d["kv_indptr"], d["kv_lens"], d["q_indptr"], d["lse"], scale,
                       d["weights"], **kw)


def reference(d, scale=C.SCALE):
    """Weights after the call, and the bounds of their errors: each term is off
    by its score's error (chunk_util) and by the roundings of the exponent (of
    scale and the logarithms' base: 2^-22 of its size) and of exp2 (2^-22); the
    sum of the block's at most rows / 4 terms in a thread and of the parts by
    2^-24 each, and the weight itself is rounded once more."""
    w, tol = d["weights"].double().numpy().copy(), np.zeros(d["weights"].shape)
    H = d["q"].shape[1]
    for b, t0, t1, n, slots, ok in C.requests(d):
        if t0 == t1:
            continue
        q, keys, lse = d["q"][t0:t1].double().numpy(), C.gather(d, slots, ok), d["lse"][t0:t1].double().numpy()
        c = t1 - t0
        rows = q.reshape(c * H, 576)
        s = scale * (rows @ keys.T)
        size = abs(scale) * (np.abs(rows) @ np.abs(keys).T)
        l = lse.reshape(-1, 1)
        gives = np.isfinite(l)
        l = np.where(gives, l, 0)
        seen = np.repeat(np.arange(n)[None] <= (n - c + np.arange(c))[:, None], H, 0) & gives & ok[None]
        e = np.where(seen, np.exp(s - l), 0)
        err = C.SCORE_STEPS * 2.0 ** -23 * size + 2.0 ** -22 * (np.abs(s) + np.abs(l) + 1)
        w[b, :n] += e.sum(0)
        tol[b, :n] = (e * np.expm1(2 * err)).sum(0) + (c * H / 256 + 80) * 2.0 ** -23 * (e.sum(0) + np.abs(w[b, :n]))
    return w, tol


def check(d, scale=C.SCALE, expect=0, **plan_kw):
    with C.plan_for(d, **plan_kw) as plan:
        g = C.to_cuda(d)
        weigh(plan, g, scale)
        torch.cuda.synchronize()
        assert plan.get_error() == expect
    compare(d, g["weights"], scale)
    return g


def compare(d, got, scale=C.SCALE):
    w, tol = reference(d, scale)
    off = np.abs(got.double().cpu().numpy() - w)
    assert (off <= tol).all(), f"{np.max(off / np.maximum(tol, 1e-300)):.3g} of the bound, {off.max():.3g}"


def test_the_oracle_of_the_sums():
    """`reference` against the loops of the definition."""
    d = make([3, 1], [10, 4], 2, 64, seed=1)
    w, _ = reference(d)
    for b, t0, t1, n, slots, ok in C.requests(d):
        add = evict_ref.weigh(d["q"][t0:t1].double().numpy(), C.gather(d, slots, ok), d["lse"][t0:t1].double().numpy(), C.SCALE)
        np.testing.assert_allclose(w[b, :n], d["weights"][b, :n].double().numpy() + add, rtol=1e-12)
        assert abs(add.sum() - (t1 - t0) * 2) < 1e-5      # every row gives 1 in all


@pytest.mark.parametrize("page", [1, 64])
@pytest.mark.parametrize("new,lens,H", [
    ([1], [1], 1),
    ([1], [2], 128),
    ([1], [257], 16),                                # a single token
    ([200], [200], 1),                               # nothing cached before
    ([65], [65], 3),
    ([130, 1], [130, 300], 20),
    ([7, 0, 3, 0], [128, 40, 260, 0], 16),           # requests without new tokens, one without rows
    ([1] * 9, [1, 64, 65, 127, 128, 129, 256, 257, 700], 64),
    ([300], [1500], 16),
    ([5, 40, 1], [500, 40, 1023], 128),
    ([3], [1000], 300),                              # more heads than a tile has rows
])
def test_matches_the_oracle(new, lens, H, page):
    check(make(new, lens, H, page, seed=sum(lens) + H))


@pytest.mark.parametrize("page", [1, 64])
def test_a_long_context(page):
    check(make([2], [20000], 32, page, seed=2))
    check(make([40, 1, 1], [9000, 3000, 500], 64, page, seed=3))


def test_blocks_that_many_clusters_share():
    check(make([400], [600], 64, 64, seed=4))
    check(make([1, 500], [10, 500], 64, 1, seed=5))
    for page in (1, 64):   # shares of a part, a whole block and a part
        check(make([8], [33000], 64, page, seed=20))
        check(make([12, 5], [20000, 13000], 64, page, seed=21))


def test_many_requests():
    check(make([i % 3 for i in range(700)], [i % 3 + i % 41 for i in range(700)], 16, 1, seed=6))


def test_scales_and_strides():
    for scale in (0.2, 1e-3, 0.0, -0.05):
        check(make([70, 9], [700, 60], 16, 64, seed=7, scale=scale), scale)
    d = make([70, 9], [700, 60], 16, 64, seed=8, extra=333)
    d["weights"] = d["weights"][:, 1::1].clone()
    with C.plan_for(d) as plan:
        g = C.to_cuda(d)
        wide = torch.full((2, 5000), 7.0, device="cuda")
        part = wide[:, 64:64 + d["weights"].shape[1]]
        part.copy_(g["weights"])
        g["weights"] = part
        weigh(plan, g)
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    compare(d, part)
    wide[:, 64:64 + d["weights"].shape[1]] = 7
    assert (wide == 7).all()


def test_calls_add_up_and_are_repeatable():
    """Two layers into the same weights; the same calls give the same bits."""
    a, b = make([60, 2], [900, 70], 32, 64, seed=9), make([60, 2], [900, 70], 32, 64, seed=10)
    got = []
    with C.plan_for(a) as plan:
        for _ in range(2):
            w = torch.zeros(2, 900, device="cuda")
            for d in (a, b):
                weigh(plan, dict(C.to_cuda(d), weights=w))
            got.append(w)
        assert plan.get_error() == 0
    assert torch.equal(*got)
    total = got[0].double().sum(1).cpu()
    assert torch.allclose(total, torch.tensor([2 * 60 * 32.0, 2 * 2 * 32.0], dtype=torch.float64), rtol=1e-5)


def test_with_the_log_sum_exps_of_the_attention():
    """What the attention's own lse is off by, its rows' weights are too: their
    sum is 1 to within both errors."""
    d = make([40, 3], [700, 90], 16, 64, seed=11)
    with C.plan_for(d) as plan:
        g = C.to_cuda(d)
        g["lse"] = C.attn(plan, g)[1]
        g["weights"].zero_()
        weigh(plan, g)
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    d["lse"], d["weights"] = g["lse"].cpu(), torch.zeros_like(d["weights"])
    compare(d, g["weights"])


def test_tokens_and_places_that_are_not_a_requests():
    d = make([5, 0, 70], [300, 40, 90], 16, 64, seed=12, front=3, pad=9, extra=20)
    for t in (0, 2, 78, 86):
        d["q"][t] = float("nan")
        d["lse"][t] = float("nan")
    g = check(d)
    for b, n in enumerate([300, 0, 90]):
        assert torch.equal(g["weights"][b, n:].cpu(), d["weights"][b, n:])


def test_rows_whose_log_sum_exp_is_not_finite_give_nothing():
    d = make([9], [300], 16, 1, seed=13)
    d["lse"][2, 3], d["lse"][4, :], d["lse"][8, 15] = float("nan"), float("-inf"), float("inf")
    d["q"][2, 3, 7] = float("nan")
    d["q"][4, 5, 500] = float("inf")
    q = d["q"].clone()
    d["q"] = torch.nan_to_num(q.float(), 0, 0, 0).bfloat16()
    want = d
    g = C.to_cuda(dict(d, q=q))
    with C.plan_for(d) as plan:
        weigh(plan, g)
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    compare(want, g["weights"])


@pytest.mark.parametrize("page", [1, 64])
def test_values_that_are_not_finite_stay_where_they_are(page):
    """A NaN row, one behind the request's last, one of a later token."""
    d = make([40, 3], [200, 70], 16, page, seed=14)
    slots = {b: s for b, _, _, _, s, _ in C.requests(d)}
    clean = dict(d, cache=d["cache"].clone())
    d["cache"][slots[0][50], 100] = float("nan")
    d["cache"][slots[0][180], 5] = float("inf")
    if page == 64:
        last = int(slots[0][199])
        d["cache"][last + 1:(last // 64 + 1) * 64] = float("nan")
    with C.plan_for(d) as plan:
        g = C.to_cuda(d)
        weigh(plan, g)
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    got = g["weights"].cpu()
    assert torch.isnan(got[0, 50]) and not torch.isfinite(got[0, 180])
    w, tol = reference(clean)
    off = np.abs(got.double().numpy() - w)
    off[0, 50] = off[0, 180] = 0
    assert (off <= tol).all()


@pytest.mark.parametrize("page", [1, 64])
def test_bad_slots_get_nothing(page):
    d = make([2, 5], [3, 200], 16, page, seed=15)
    d["kv_indices"][0] = -1
    if page == 1:
        d["kv_indices"][1:3] = torch.tensor([d["cache"].shape[0], 1 << 30], dtype=torch.int32)
        d["kv_indices"][50] = -7
    else:
        d["kv_indices"][2] = d["cache"].shape[0] // 64
    d["lse"].fill_(5.0)
    g = check(d, expect=mb.DEV_BAD_SLOT)
    assert torch.equal(g["weights"][0].cpu(), d["weights"][0])


@pytest.mark.parametrize("batch", [4, 700])
def test_requests_that_cannot_be_served_are_left_alone(batch):
    new, lens = [9, 2, 30, 4] + [1] * (batch - 4), [100, 40, 30, 70] + [3] * (batch - 4)
    good = make(new, lens, 16, 64, seed=16, pad=2)
    for name, at, value, bit in (("kv_lens", 1, 1, mb.DEV_BAD_LEN), ("kv_lens", 1, 101, mb.DEV_BAD_LEN),
                                 ("kv_lens", 1, -5, mb.DEV_BAD_LEN), ("kv_indptr", 2, 1, mb.DEV_BAD_INDPTR)):
        d = dict(good)
        d[name] = good[name].clone()
        d[name][at] = value
        with C.plan_for(good) as plan:
            g = C.to_cuda(d)
            weigh(plan, g)
            torch.cuda.synchronize()
            assert plan.get_error() == bit
        got = g["weights"].cpu()
        w, tol = reference(good)
        out = [1, 2] if name == "kv_indptr" else [1]
        assert torch.equal(got[out], good["weights"][out])
        rest = [b for b in range(batch) if b not in out]
        assert (np.abs(got.double().numpy() - w)[rest] <= tol[rest]).all()


@pytest.mark.parametrize("tokens", [[0, 9, 8, 41, 45], [-1, 9, 11, 41, 45], [0, 9, 11, 41, 48]])
def test_tokens_that_are_not_divided_add_nothing(tokens):
    d = make([9, 2, 30, 4], [100, 40, 30, 70], 16, 1, seed=17)
    with C.plan_for(d) as plan:
        g = C.to_cuda(d)
        g["q_indptr"] = torch.tensor(tokens, dtype=torch.int32, device="cuda")
        weigh(plan, g)
        torch.cuda.synchronize()
        assert plan.get_error() == mb.DEV_BAD_INDPTR
    assert torch.equal(g["weights"].cpu(), d["weights"])


def test_captured_and_replayed_and_on_another_stream():
    d = make([40, 1, 1], [700, 300, 64], 16, 64, seed=18, pad=3)
    with C.plan_for(d) as plan:
        g = C.to_cuda(d)
        eager = dict(g, weights=g["weights"].clone())
        weigh(plan, eager)
        side = torch.cuda.Stream()
        other = dict(g, weights=g["weights"].clone())
        torch.cuda.synchronize()
        weigh(plan, other, stream=side)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            weigh(plan, g)
        graph.replay()
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    assert torch.equal(g["weights"], eager["weights"]) and torch.equal(other["weights"], eager["weights"])
    compare(d, g["weights"])


@pytest.mark.parametrize("page", [1, 64])
@pytest.mark.parametrize("fault", [mb.FAULT_EVEN_GIVES_UP, mb.FAULT_ODD_GIVES_UP])
@pytest.mark.parametrize("new,lens,H", [([1] * 40, [1500] * 40, 16), ([40], [9000], 64)])
def test_weights_of_a_pair_that_gave_up_are_nan(new, lens, H, fault, page):
    """One CTA of each pair stops in its second step, the other's waits run out:
    a weight is NaN, or right where its block was done before or is shared with
    nobody who stopped.  The next call is right."""
    d = make(new, lens, H, page, seed=22)
    with C.plan_for(d) as plan:
        g = C.to_cuda(d)
        plan.inject_fault(fault)
        weigh(plan, g)
        torch.cuda.synchronize()
        assert plan.get_error() == mb.DEV_TIMEOUT
        got = g["weights"].double().cpu().numpy()
        w, tol = reference(d)
        lost = np.isnan(got)
        assert lost.mean() > 0.5 and (lost | (np.abs(np.where(lost, 0, got) - w) <= tol)).all()
        g = C.to_cuda(d)
        weigh(plan, g)
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    compare(d, g["weights"])


def test_no_tokens_and_refusals():
    d = make([2, 1], [70, 5], 16, 64, seed=19)
    g = C.to_cuda(d)
    with C.plan_for(d) as plan:
        weigh(plan, dict(g, q=g["q"][:0], lse=g["lse"][:0]))
        assert torch.equal(g["weights"].cpu(), d["weights"])
        for bad in (dict(g, q=g["q"].float()), dict(g, cache=g["cache"][:-64]), dict(g, lse=g["lse"].double()),
                    dict(g, lse=g["lse"][:2]), dict(g, weights=g["weights"][:, :-1]), dict(g, weights=g["weights"][:1]),
                    dict(g, weights=g["weights"].double()), dict(g, weights=g["weights"].cpu()),
                    dict(g, weights=torch.zeros(70, 2, device="cuda").t()), dict(g, weights=torch.zeros(1, 70, device="cuda").expand(2, 70)),
                    dict(g, q_indptr=g["q_indptr"][:2])):
            with pytest.raises((TypeError, ValueError)):
                weigh(plan, bad)
        with pytest.raises(mb.MlaVerifyError):
            weigh(plan, g, scale=float("inf"))
        with pytest.raises(mb.MlaVerifyError):          # rows that do not begin on 16 bytes
            weigh(plan, dict(g, weights=torch.zeros(2, 80, device="cuda")[:, 1:72]))
        lib = mb.load_library()
        p = lambda x: x.data_ptr()  # noqa: E731
        args = [p(g[k]) for k in ("q", "cache", "kv_indices", "kv_indptr", "kv_lens", "q_indptr", "lse")]
        assert lib.mla_verify_weigh_kv(plan.handle, 3, 3, *args, 1.0, p(g["weights"]), 70, None) == -4
        for n, stride in ((-1, 70), ((1 << 31) // 16, 70), (1 << 62, 70), (3, 69), (3, 1 << 62)):
            assert lib.mla_verify_weigh_kv(plan.handle, 2, n, *args, 1.0, p(g["weights"]), stride, None) == -9
        for i in range(7):
            assert lib.mla_verify_weigh_kv(plan.handle, 2, 3, *(a if k != i else None for k, a in enumerate(args)), 1.0,
                                           p(g["weights"]), 70, None) == -1
        assert lib.mla_verify_weigh_kv(plan.handle, 2, 3, *args, 1.0, None, 70, None) == -1
        torch.cuda.synchronize()
        assert plan.get_error() == 0
