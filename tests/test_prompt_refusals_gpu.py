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


def _fork(plan, layers, stride):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = torch.zeros(3 * 512, 576, dtype=torch.bfloat16, device="cuda")
    t = [i32([0]), i32([3, 1]), i32([0, 2]), i32([100])]
    pool = [i32([0, 1, 0, 1, 0, 0, 0, 0]), i32([0, 2, 4, 5, 6, 7, 0, 0]), i32([6])]
    out = [i32([-1] * 8), i32([-1, -1]), i32([-1])]
    p = lambda x: x.data_ptr()  # noqa: E731
    st = mb.load_library().mla_verify_fork_kv(plan.handle, 1, p(t[0]), 1, p(t[1]), p(t[2]), p(t[3]), p(cache), layers, stride, 0,
                                              *map(p, pool), p(out[0]), 8, p(out[1]), p(out[2]), None)
    torch.cuda.synchronize()
    return st, int(pool[2])


def test_layers_that_overlap_or_are_too_many():
    size = 512 * 576
    with mb.Plan(2, 1, 1, 64, 512, 256) as plan:
        for layers, stride in ((2, 0), (2, size - 8), (3, 64 * 576), (1 << 16, 0), ((1 << 16) + 1, size), ((1 << 31) - 1, size)):
            assert _fork(plan, layers, stride) == (-9, 6), (layers, stride)
        for layers, stride in ((1, 0), (1, 8), (2, size), (3, size)):
            assert _fork(plan, layers, stride) == (0, 5)
        assert plan.get_error() == 0


def test_a_cache_whose_layers_are_one():
    """Layers of a broadcast cache lie on one another: refused, too."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = torch.zeros(512, 576, dtype=torch.bfloat16, device="cuda")
    with mb.Plan(2, 1, 1, 64, 512, 256) as plan:
        with pytest.raises(mb.MlaVerifyError):
            mb.fork_kv(plan, i32([0]), i32([3, 1]), i32([0, 2]), i32([100]), cache.expand(2, 512, 576), i32([0] * 8), i32([0] * 8),
                       i32([6]))
