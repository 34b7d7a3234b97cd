"""Outputs that a call allocates itself, on another stream than the current one."""
import pytest
import torch

from paged_mla_speculative_gb300 import binding as mb
from tests import gpu_util as G
from tests.test_append_gpu import _case
from tests.test_shared_gpu import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def _late_reader_keeps_its_input(shape, dtype, call):
    """A tensor of `shape` is freed on the current stream while a copy of it is
    still queued there (behind a bounded ~50 ms kernel); `call` then allocates
    as much for another stream.  The copy must not see the call's output."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for stream in (side, side.cuda_stream):          # a torch stream, and a raw handle
        x = torch.full(shape, 7, dtype=dtype, device="cuda")
        y = torch.empty_like(x)
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        y.copy_(x)
        del x
        call(stream)
        torch.cuda.synchronize()
        assert (y == 7).all()


def test_append_queries():
    N, H = 64, 32
    d = {k: v.cuda() for k, v in _case(N, H, seed=1).items()}
    with mb.Plan(1, 1, H, 1, 256, 64) as plan:
        _late_reader_keeps_its_input((N, H, 576), torch.bfloat16, lambda s: mb.append_kv(
            plan, d["kv"], d["weight"], 1e-6, d["cos_sin"], d["positions"], d["slots"], d["kv_cache"], q_nope=d["q_nope"],
            q_pe=d["q_pe"], stream=s))


def test_shared_attention():
    inp, gp, sl = make([2], [256], [7, 20], 8, 64, seed=2)
    d, gp, sl = G.to_cuda(inp), gp.cuda(), sl.cuda()
    with G.make_plan(inp) as plan:
        _late_reader_keeps_its_input((2, 8, 64, 512), torch.float32, lambda s: mb.mla_verify_attn_shared(
            plan, d.q, d.kv_cache, d.kv_indices, d.kv_indptr, d.kv_lens, d.draft_parent, d.scale, gp, sl, stream=s))


def test_forked_tables():
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pages, kids = 64, 16
    cache = torch.zeros(pages * 64, 576, dtype=torch.bfloat16, device="cuda")
    with mb.Plan(kids, 1, 1, 64, pages * 64, 64 * 1024) as plan:
        refs, free, count = i32([0] * pages), i32(list(range(8, pages)) + list(range(8))), i32([pages])
        parents, idx, ptr, lens = i32([0] * kids), i32([0]), i32([0, 0]), i32([0])   # a parent without rows
        _late_reader_keeps_its_input((kids * 1024,), torch.int32, lambda s: mb.fork_kv(
            plan, parents, idx, ptr, lens, cache, refs, free, count, extra_rows=128, stream=s))
        assert plan.get_error() == 0 and int(count) == 0
