"""Numerics of the shared-prefix verify attention where the weights of a row
span more than fp16 does, against the fp64 oracle, by relative error.

Tolerance of an output whose value parts are all positive: P^T is rounded to
fp16 once (2^-11 of each weight, and all equal weights alike); the scores here
are exact, their exponents lose 2^-20 at most, and the fp32 sums of a cluster's
few thousand keys less than 2^-14.
"""
import dataclasses

import numpy as np
import pytest
import torch

from paged_mla_speculative_gb300 import binding as mb
from tests import gpu_util as G
from tests.test_shared_gpu import make, run

pytestmark = pytest.mark.gpu

REL = 2.0 ** -11 + 2.0 ** -14


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def _one_dim_scores(shared, sink, others, q0, T=4, H=16, seed=60):
    """Two requests whose scores come from rope dim 0 alone: the first shared
    key has `sink` there and a value part of zeros, every other key `others`
    and values in [0.5, 1.5); head h of every draft has q0[h]."""
    inp, gp, sl = make([2], [shared], [9, 40], T, H, seed=seed, spike_frac=0.0)
    g = torch.Generator().manual_seed(seed)
    cache = torch.zeros_like(inp.kv_cache)
    cache[:, :512] = (0.5 + torch.rand(cache.shape[0], 512, generator=g)).to(torch.bfloat16)
    cache[:, 512] = others
    first = int(inp.kv_indices[0])
    cache[first] = 0
    cache[first, 512] = sink
    q = torch.zeros_like(inp.q)
    q[..., 512] = torch.tensor(q0, dtype=torch.float32).to(torch.bfloat16)
    return dataclasses.replace(inp, q=q, kv_cache=cache), gp, sl


@pytest.mark.parametrize("shared", [600, 40000])     # a whole tile; parts of one merged
def test_a_dominant_key_without_value(shared):
    """One key up to 17.4 nats ahead (its weight is 2^25 times another's) holds
    no value: the output is what the others' small weights add up to."""
    case = _one_dim_scores(shared, 15.0625, 0.0, [16.0 - 0.5 * h for h in range(16)])
    with G.make_plan(case[0]) as plan:
        out, lse = run(plan, *case)
        assert plan.get_error() == 0
    ro, rl = G.oracle_full(case[0])
    assert ro.min() > 0
    assert (np.abs(out.double().cpu().numpy() - ro) <= REL * ro).all()
    assert (np.abs(lse.double().cpu().numpy() - rl) <= 2.0 ** -16 * np.maximum(1, np.abs(rl))).all()


@pytest.mark.parametrize("sink,others", [(59904.0, 0.0), (0.0, 59904.0), (59904.0, 59904.0), (59904.0, -59904.0)])
def test_scores_beyond_the_exactness_of_fp32(sink, others):
    """Scores up to 3e8: every weight is 1 or 0, of the smallest query 2^-40."""
    q0 = [s * v for v in (59904.0, 40192.0, 3008.0, 520.0, 260.0, 130.0, 65.0, 2.0 ** -16) for s in (1.0, -1.0)]
    case = _one_dim_scores(300, sink, others, q0)
    with G.make_plan(case[0]) as plan:
        out, lse = run(plan, *case)
        assert plan.get_error() == 0
    ro, rl = G.oracle_full(case[0])
    assert (np.abs(out.double().cpu().numpy() - ro) <= REL * np.abs(ro)).all()
    # the scaled score is rounded in units of log2 and again as lse
    assert (np.abs(lse.double().cpu().numpy() - rl) <= 2.0 ** -21 * np.maximum(1, np.abs(rl)) + 2.0 ** -16).all()


@pytest.mark.parametrize("exponent", [-10, -18, -22, -27])
def test_small_values_and_queries(exponent):
    """bf16 holds magnitudes that fp16 does not: a key or query value keeps an
    absolute error of 2^-25 (none from 2^-14 on), and one below that becomes 0.
    Outputs are off by as much beside the rounding of P^T; scores by 2^-25 times
    the 1-norm of the other side (below 576 * 4) and by the 36 fp32 additions of
    16 products each, 2^-23 of a sum that is below 200 before the scale of 0.07."""
    small = 2.0 ** exponent
    inp, gp, sl = make([2], [900], [9, 40], 4, 16, seed=61, spike_frac=0.0)
    cache = inp.kv_cache.clone()
    cache[:, :512] = (cache[:, :512].float() * small).to(torch.bfloat16)
    q = inp.q.clone()
    q[:, 2:] = (q[:, 2:].float() * small).to(torch.bfloat16)
    for case in ((dataclasses.replace(inp, kv_cache=cache), gp, sl), (dataclasses.replace(inp, q=q), gp, sl)):
        with G.make_plan(case[0]) as plan:
            out, lse = run(plan, *case)
            assert plan.get_error() == 0
        ro, rl = G.oracle_full(case[0])
        big = float(case[0].kv_cache[case[0].kv_indices.long(), :512].double().abs().max())   # (other rows hold NaN)
        score = (2.0 ** -25 * 576 * 4 + 36 * 2.0 ** -23 * 200) * abs(case[0].scale)
        assert (np.abs(lse.double().cpu().numpy() - rl) <= score + 2.0 ** -20).all()
        assert (np.abs(out.double().cpu().numpy() - ro) <= 2.0 ** -25 + (2.0 ** -11 + 2 * score + 2.0 ** -14) * big).all()


@pytest.mark.parametrize("scale", [-0.07, 0.0, -0.0, 1e-30])
def test_negative_and_vanishing_scales(scale):
    inp, gp, sl = make([2, 1], [600, 100], [9, 300, 40], 4, 16, seed=62, spike_frac=0.0)
    case = (dataclasses.replace(inp, scale=scale), gp, sl)
    with G.make_plan(inp) as plan:
        out, lse = run(plan, *case)
        assert plan.get_error() == 0
    G.assert_parity(out.cpu().numpy(), lse.cpu().numpy(), *G.oracle_full(case[0]))
