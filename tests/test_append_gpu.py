"""New tokens' cache rows and queries on the GPU against the fp64 oracle.

Tolerance: every element is rounded to bf16 once (2^-8 of its magnitude at
most).  Before that the latent passes a 512-term fp32 sum of squares, a
reciprocal root and two products: well under 2^-16 of its magnitude.  A
rotated element is two products and a sum in fp32: 3 * 2^-24 of the two
terms' magnitudes.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle.append_ref as ar
from paged_mla_speculative_gb300 import binding as mb

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def _table(max_pos):
    t = torch.arange(max_pos, dtype=torch.float64)
    angle = t[:, None] * 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    return torch.cat((angle.cos(), angle.sin()), -1).float()


def _case(N, H, seed, slots=256, max_pos=500):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g).to(BF)  # noqa: E731
    return dict(kv=rand(N, 576) * 3, weight=(1 + 0.3 * torch.randn(512, generator=g)).to(BF), q_nope=rand(N, H, 512),
                q_pe=rand(N, H, 64), cos_sin=_table(max_pos), positions=torch.randint(0, max_pos, (N,), generator=g).int(),
                slots=torch.randperm(slots, generator=g)[:N].int(), kv_cache=rand(slots, 576), q=rand(N, H, 576))


def _check(c, cache, q, halves, eps=1e-6, nope=True):
    n64 = {k: v.double().numpy() for k, v in c.items()}
    ref_c, ref_q, flags = ar.append_kv(n64["kv"], n64["weight"], eps, n64["q_nope"] if nope else None, n64["q_pe"],
                                       n64["cos_sin"], c["positions"].tolist(), c["slots"].tolist(), halves,
                                       n64["kv_cache"], n64["q"])
    big = np.abs(n64["kv"][:, 512:]).max(initial=0) + np.abs(n64["q_pe"]).max(initial=0)
    for got, ref in ((cache, ref_c), (q, ref_q)):
        got = got.double().cpu().numpy()
        assert (np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(ref) + 4 * 2.0 ** -24 * big).all()
    # nothing else was written
    untouched = np.ones(len(n64["kv_cache"]), bool)
    good = [s for s, p in zip(c["slots"].tolist(), c["positions"].tolist())
            if 0 <= s < len(untouched) and 0 <= p < len(c["cos_sin"])]
    untouched[good] = False
    assert np.array_equal(cache.cpu().double().numpy()[untouched], n64["kv_cache"][untouched])
    return flags


def _run(plan, c, halves, **over):
    d = {k: v.cuda() for k, v in c.items()}
    d.update(over)
    mb.append_kv(plan, d["kv"], d["weight"], 1e-6, d["cos_sin"], d["positions"], d["slots"], d["kv_cache"],
                 q_nope=d["q_nope"], q_pe=d["q_pe"], q=d["q"], interleaved=not halves)
    torch.cuda.synchronize()
    return d["kv_cache"], d["q"]


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("N,H", [(1, 1), (1, 16), (7, 3), (64, 20), (130, 5)])
def test_matches_the_oracle(N, H, halves):
    c = _case(N, H, seed=N + H)
    with mb.Plan(1, 1, H, 1, 256, 64) as plan:
        cache, q = _run(plan, c, halves)
        assert _check(c, cache, q, halves) == plan.get_error() == 0


def test_padding_bad_slots_and_bad_positions_write_nothing():
    c = _case(9, 6, seed=3)
    c["slots"][1] = c["slots"][8] = -1
    c["slots"][2], c["slots"][3] = 256, -5
    c["positions"][4], c["positions"][5] = 500, -1
    with mb.Plan(1, 1, 6, 1, 256, 64) as plan:
        cache, q = _run(plan, c, False)
        assert _check(c, cache, q, False) == plan.get_error() == mb.DEV_BAD_SLOT | mb.DEV_BAD_POS
        c["slots"][:] = -1
        cache, q = _run(plan, c, False)
        assert torch.equal(cache.cpu(), c["kv_cache"]) and torch.equal(q.cpu(), c["q"]) and plan.get_error() == 0


def test_slices_of_wider_tensors_and_rotation_in_place():
    N, H = 33, 7
    c = _case(N, H, seed=8)
    fused = torch.zeros(N, 24 + 576, dtype=BF).cuda()
    fused[:, 24:] = c["kv"].cuda()
    wide = torch.zeros(H, N, 128 + 64, dtype=BF).cuda()           # heads outermost
    wide[..., 128:] = c["q_pe"].transpose(0, 1).cuda()
    with mb.Plan(1, 1, H, 1, 256, 64) as plan:
        cache, q = _run(plan, c, True, kv=fused[:, 24:], q_pe=wide.transpose(0, 1)[..., 128:])
        _check(c, cache, q, True)
        # one absorbed vector for all heads, by a stride of 0
        one = c["q_nope"][:, :1].cuda()
        cache, q = _run(plan, c, True, q_nope=one.expand(N, H, 512))
        _check({**c, "q_nope": c["q_nope"][:, :1].expand(N, H, 512)}, cache, q, True)
        for halves in (False, True):   # q holds everything already
            c2 = {**c, "q_pe": c["q"][..., 512:]}
            d = c["q"].cuda()
            cache, q = _run(plan, c2, halves, q=d, q_pe=d[..., 512:], q_nope=None)
            _check(c2, cache, q, halves, nope=False)
        # keys alone, and no token at all
        d = {k: v.cuda() for k, v in c.items()}
        assert mb.append_kv(plan, d["kv"], d["weight"], 1e-6, d["cos_sin"], d["positions"], d["slots"], d["kv_cache"]) is None
        torch.cuda.synchronize()
        _check(c, d["kv_cache"], _run(plan, c, False)[1], False)
        e = {k: d[k][:0] for k in ("kv", "positions", "slots")}
        before = d["kv_cache"].clone()
        mb.append_kv(plan, e["kv"], d["weight"], 1e-6, d["cos_sin"], e["positions"], e["slots"], d["kv_cache"])
        torch.cuda.synchronize()
        assert torch.equal(before, d["kv_cache"]) and plan.get_error() == 0


def test_extreme_values():
    """Zero and huge latents: eps keeps a zero row finite; 3e18^2 * 512 stays
    inside fp32; infinities and NaN stay in their own token."""
    c = _case(5, 4, seed=11)
    c["kv"][0] = 0
    c["kv"][1, :512] = 3e17
    c["kv"][2, 5] = float("nan")
    c["q_pe"][3, 2, 7] = float("inf")
    with mb.Plan(1, 1, 4, 1, 256, 64) as plan:
        cache, q = _run(plan, c, False)
    s = c["slots"].long()
    assert (cache[s[0]] == 0).all()
    assert torch.isnan(cache[s[2], :512]).all() and torch.isfinite(cache[s[2], 512:]).all()
    assert torch.isfinite(q[3, :2]).all() and torch.isfinite(q[3, 3]).all() and not torch.isfinite(q[3, 2, 518:520]).any()
    keep = [1, 4]
    sub = {k: (v[keep] if k in ("kv", "q_nope", "q_pe", "positions", "slots", "q") else v) for k, v in c.items()}
    rest = c["kv_cache"].clone()
    rest[s[keep]] = cache[s[keep]].cpu()
    _check(sub, rest, q[keep], False)


def test_rows_beyond_the_32_bit_offset():
    slots = (1 << 22) + 64                       # 2.4e9 elements
    c = _case(3, 2, seed=5)
    place = torch.tensor([slots - 1, 3, 3_800_000], dtype=torch.int32)
    cache = torch.zeros(slots, 576, dtype=BF, device="cuda")
    with mb.Plan(1, 1, 2, 1, slots, 64) as plan:
        _run(plan, c, False, slots=place.cuda(), kv_cache=cache)
        assert plan.get_error() == 0
    small = {**c, "slots": torch.tensor([0, 1, 2]).int(), "kv_cache": torch.zeros(3, 576, dtype=BF)}
    _check(small, cache[place.long().cuda()], _run_q(c), False)
    assert int((cache != 0).any(1).sum()) == 3


def _run_q(c):
    with mb.Plan(1, 1, c["q"].shape[1], 1, 256, 64) as plan:
        return _run(plan, c, False)[1]


def test_captured_and_replayed_on_another_stream():
    H = 8
    cases = [_case(20, H, seed=s) for s in (1, 2)]
    cases[1]["slots"][15:] = -1
    d = {k: v.cuda() for k, v in cases[0].items()}
    with mb.Plan(1, 1, H, 1, 256, 64) as plan:
        s = torch.cuda.Stream()
        call = lambda: mb.append_kv(plan, d["kv"], d["weight"], 1e-6, d["cos_sin"], d["positions"], d["slots"],  # noqa: E731
                                    d["kv_cache"], q_nope=d["q_nope"], q_pe=d["q_pe"], q=d["q"], stream=s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
        for c in cases:
            for k, v in c.items():
                d[k].copy_(v)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            _check(c, d["kv_cache"], d["q"], False)
        assert plan.get_error() == 0


def test_host_argument_errors():
    d = {k: v.cuda() for k, v in _case(4, 2, seed=1).items()}
    with mb.Plan(1, 1, 2, 1, 256, 64) as plan:
        lib = mb.load_library()

        def call(**k):
            a = dict(n=4, kv=d["kv"].data_ptr(), ks=576, w=d["weight"].data_ptr(), eps=1e-6, nope=d["q_nope"].data_ptr(),
                     ns=1024, nh=512, pe=d["q_pe"].data_ptr(), ps=128, ph=64, cs=d["cos_sin"].data_ptr(), mp=500,
                     pos=d["positions"].data_ptr(), slots=d["slots"].data_ptr(), style=0, cache=d["kv_cache"].data_ptr(),
                     q=d["q"].data_ptr())
            a.update(k)
            return lib.mla_verify_append_kv(plan.handle, a["n"], a["kv"], a["ks"], a["w"], ctypes.c_float(a["eps"]), a["nope"],
                                            a["ns"], a["nh"], a["pe"], a["ps"], a["ph"], a["cs"], a["mp"], a["pos"], a["slots"],
                                            a["style"], a["cache"], a["q"], None)
        assert call() == 0 and call(n=0, kv=None) == 0 and call(pe=None, q=None, nope=None) == 0
        for k in ("kv", "w", "cs", "pos", "slots", "cache", "q"):
            assert call(**{k: None}) == -1, k
        for k in ("kv", "w", "cs", "pos", "slots", "cache", "q", "pe", "nope"):
            assert call(**{k: d["q"].data_ptr() + 8}) == -2, k
        for bad in (dict(n=-1), dict(mp=0), dict(ks=580), dict(ns=-8), dict(nh=4), dict(ps=1), dict(ph=-64), dict(style=2),
                    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
            assert call(**bad) == -9, bad
        torch.cuda.synchronize()
        assert plan.get_error() == 0
