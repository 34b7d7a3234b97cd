"""Requests without new tokens, as the idle slots of a captured batch are: their
lengths and tables, whatever they hold, are not looked at."""
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


STALE = [0, 20, 100, -5, 9999, 1 << 30]   # none is the length that the idle requests' tables were made for


def idle_among(batch, page, **kw):
    """Inputs of `batch` requests, every other one idle with 40 rows."""
    return TW.make([(5, 0, 3, 0)[b % 4] for b in range(batch)], [(70, 40, 130, 40)[b % 4] for b in range(batch)], 16, page, seed=batch, **kw)


def with_lengths(g, length):
    """`g` with `length` for the idle requests'."""
    lens = g["kv_lens"].clone()
    lens[1::2] = length
    return dict(g, kv_lens=lens)


@pytest.mark.parametrize("page", [1, 64])
@pytest.mark.parametrize("batch", [4, 30, 600])
def test_chunks_beside_idle_requests(batch, page):
    d = idle_among(batch, page)
    g = C.to_cuda(d)
    with C.plan_for(d) as plan:
        out, lse = C.attn(plan, g)
        C.assert_close(d, out, lse)
        for length in STALE:
            again = C.attn(plan, with_lengths(g, length))
            torch.cuda.synchronize()
            assert plan.get_error() == 0, length
            assert torch.equal(again[0], out) and torch.equal(again[1], lse), length


@pytest.mark.parametrize("batch", [4, 600])
def test_chunks_beside_released_tables(batch):
    """Idle requests whose pages were given back: empty tables, lengths as they were."""
    d = C.make([(5, 0, 3, 0)[b % 4] for b in range(batch)], [(70, 0, 130, 0)[b % 4] for b in range(batch)], 16, 64, seed=batch)
    with C.plan_for(d) as plan:
        out, lse = C.attn(plan, with_lengths(C.to_cuda(d), 40))
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    C.assert_close(d, out, lse)


@pytest.mark.parametrize("page", [1, 64])
@pytest.mark.parametrize("batch", [4, 30, 900])
def test_weights_beside_idle_requests(batch, page):
    d = idle_among(batch, page, extra=20)
    g = C.to_cuda(d)
    with C.plan_for(d) as plan:
        first = dict(g, weights=g["weights"].clone())
        TW.weigh(plan, first)
        TW.compare(d, first["weights"])
        assert torch.equal(first["weights"][1::2], g["weights"][1::2])
        for length in STALE:
            again = with_lengths(dict(g, weights=g["weights"].clone()), length)
            TW.weigh(plan, again)
            torch.cuda.synchronize()
            assert plan.get_error() == 0, length
            assert torch.equal(again["weights"], first["weights"]), length
