"""The norm of latents over bf16's whole range, against the fp64 oracle.

Tolerance: as for ordinary rows -- one rounding to bf16 (2^-8), and before it
fp32 sums, a reciprocal root and two products (2^-16); results below bf16's
normal range lose their last bits absolutely (2^-133).
"""
import numpy as np
import pytest
import torch

import oracle.append_ref as ar
from paged_mla_speculative_gb300 import binding as mb
from tests.test_append_gpu import _case

pytestmark = pytest.mark.gpu

BIG = float(torch.finfo(torch.bfloat16).max)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


@pytest.mark.parametrize("eps", [1e-6, 1e-30, 0.0])
def test_rows_of_every_magnitude(eps):
    c = _case(14, 2, seed=21)
    kv = c["kv"]
    for n, scale in enumerate((1e17, 3e18, 1e25, 1e36, 1e-10, 1e-15, 1e-21, 1e-30, 1e-37)):
        kv[n, :512] = (kv[n, :512].float() * scale).to(torch.bfloat16)
    kv[9, :512] = BIG                                # every element the largest
    kv[10, 7] = 1e30                                 # one element far above the others
    kv[11, :512] = 1e-30
    kv[11, 3] = 1e-20
    kv[12, :512] = 1e-40                             # below bf16's normal range
    kv[13, 100] = -BIG
    d = {k: v.cuda() for k, v in c.items()}
    with mb.Plan(1, 1, 2, 1, 256, 64) as plan:
        mb.append_kv(plan, d["kv"], d["weight"], eps, d["cos_sin"], d["positions"], d["slots"], d["kv_cache"])
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    n64 = {k: v.double().numpy() for k, v in c.items()}
    want, _, _ = ar.append_kv(n64["kv"], n64["weight"], float(np.float32(eps)), None, np.zeros((14, 0, 64)), n64["cos_sin"],
                              c["positions"].tolist(), c["slots"].tolist(), False, n64["kv_cache"], np.zeros((14, 0, 576)))
    got = d["kv_cache"].double().cpu().numpy()
    for n, s in enumerate(c["slots"].tolist()):
        off = np.abs(got[s, :512] - want[s, :512])
        assert (off <= (2.0 ** -8 + 2.0 ** -16) * np.abs(want[s, :512]) + 2.0 ** -133).all(), n
    rest = np.ones(256, bool)
    rest[c["slots"].tolist()] = False
    assert np.array_equal(got[rest], n64["kv_cache"][rest])
