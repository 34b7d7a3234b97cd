"""Requests without new tokens, as the idle slots of a captured batch are: their
lengths and tables, whatever they hold, are not looked at."""
import numpy as np
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


def idle_among(batch, page, length, **kw):
    """Inputs of `batch` requests, every other one idle, and the same with `length`
    in the place of the idle ones' 40 rows."""
    new = [(5, 0, 3, 0)[b % 4] for b in range(batch)]
    lens = [(70, 40, 130, 40)[b % 4] for b in range(batch)]
    good = TW.make(new, lens, 16, page, seed=batch, **kw)
    stale = dict(good, kv_lens=good["kv_lens"].clone())
    stale["kv_lens"][[b for b in range(batch) if new[b] == 0]] = length
    return good, stale


@pytest.mark.parametrize("page", [1, 64])
@pytest.mark.parametrize("batch", [4, 30, 600])
@pytest.mark.parametrize("length", STALE)
def test_chunks_beside_idle_requests(length, batch, page):
    good, stale = idle_among(batch, page, length)
    with C.plan_for(good) as plan:
        out, lse = C.attn(plan, C.to_cuda(stale))
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    C.assert_close(good, out, lse)


@pytest.mark.parametrize("batch", [4, 600])
def test_chunks_beside_released_tables(batch):
    """Idle requests whose pages were given back: empty tables, lengths as they were."""
    new = [(5, 0, 3, 0)[b % 4] for b in range(batch)]
    good = C.make(new, [(70, 0, 130, 0)[b % 4] for b in range(batch)], 16, 64, seed=batch)
    stale = dict(good, kv_lens=good["kv_lens"].clone())
    stale["kv_lens"][1::2] = 40
    with C.plan_for(good) as plan:
        out, lse = C.attn(plan, C.to_cuda(stale))
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    C.assert_close(good, out, lse)
