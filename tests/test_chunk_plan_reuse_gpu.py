"""One plan for chunk calls of all sizes in a row, the one that fills its batch
and its key space before and behind the small ones."""
import pytest
import torch

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
def test_the_largest_call_around_small_ones(page):
    sizes = [([1] * 8, [2000] * 8), ([1], [70]), ([50, 9, 20], [2000, 700, 300]), ([300], [1900]), ([2, 2, 2], [500, 2, 64])]
    calls = [TW.make(new, lens, 16, page, seed=sum(lens), extra=2000 - max(lens)) for new, lens in sizes]
    slots = max(d["cache"].shape[0] for d in calls)
    for d in calls:
        d["cache"] = torch.cat((d["cache"], torch.zeros(slots - d["cache"].shape[0], 576).bfloat16()))
    first = calls[0]
    with C.plan_for(first, max_batch=8, max_kv_len=2000) as plan:
        for d in [*calls, first]:
            g = C.to_cuda(d)
            out, lse = C.attn(plan, g)
            TW.weigh(plan, g)
            torch.cuda.synchronize()
            assert plan.get_error() == 0
            C.assert_close(d, out, lse)
            TW.compare(d, g["weights"])
