"""The shared-prefix verify attention when a wait runs out: a CTA of every pair
stops in mid-call (injected on the host), the waits of its peer run out after
their cycle limit (about a second).  Every row of the pair is NaN, whichever
of the two gave up, the status word says so, and the next call is right."""
import pytest
import torch

from paged_mla_speculative_gb300 import binding as mb
from tests import gpu_util as G
from tests.test_shared_gpu import make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fault", [mb.FAULT_EVEN_GIVES_UP, mb.FAULT_ODD_GIVES_UP])
@pytest.mark.parametrize("sizes,shared,own,T,H", [
    ([8], [9000], [9, 100, 3, 0, 50, 7, 1, 2], 8, 64),                # every tile cut into parts
    ([1] * 40, [700] * 40, [i % 7 for i in range(40)], 2, 64),        # whole tiles, one per pair
    ([1] * 90, [800] * 90, [i % 50 for i in range(90)], 1, 128),      # several tiles per pair, some finished before
])
def test_every_row_of_a_pair_that_gave_up_is_nan(sizes, shared, own, T, H, fault, out_dtype):
    case = make(sizes, shared, own, T, H, seed=70)
    with G.make_plan(case[0], out_dtype) as plan:
        plan.inject_fault(fault)
        out, lse = run(plan, *case)
        assert plan.get_error() == mb.DEV_TIMEOUT
        assert torch.isnan(out).all() and torch.isnan(lse).all()
        out, lse = run(plan, *case)
        assert plan.get_error() == 0
    ref_o, ref_l = G.oracle_full(case[0])
    if out_dtype == torch.float32:
        G.assert_parity(out.cpu().numpy(), lse.cpu().numpy(), ref_o, ref_l)
    else:
        G.assert_bf16_parity(out.cpu(), lse.cpu().numpy(), ref_o, ref_l)
