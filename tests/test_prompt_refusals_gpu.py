"""Sizes that the shared-prompt calls refuse on the host, before any launch."""
import pytest
import torch

from paged_mla_speculative_gb300 import binding as mb
from tests.test_append_gpu import _case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


@pytest.mark.parametrize("n", [1 << 31, 1 << 59, 1 << 62, (1 << 63) - 1])
def test_more_tokens_than_there_can_be(n):
    """(At 2^59 tokens of 64 heads the count of work items would pass 64 bits.)"""
    d = {k: v.cuda() for k, v in _case(4, 64, seed=1).items()}
    with mb.Plan(1, 1, 64, 1, 256, 64) as plan:
        st = mb.load_library().mla_verify_append_kv(
            plan.handle, n, d["kv"].data_ptr(), 576, d["weight"].data_ptr(), 1e-6, None, 0, 0, d["q_pe"].data_ptr(), 64 * 64, 64,
            d["cos_sin"].data_ptr(), 500, d["positions"].data_ptr(), d["slots"].data_ptr(), 0, d["kv_cache"].data_ptr(),
            d["q"].data_ptr(), None)
        assert st == -9
        torch.cuda.synchronize()
        assert plan.get_error() == 0
