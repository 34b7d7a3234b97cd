"""evict_kv refuses outputs that lie in its inputs or in one another, wherever
they begin, and takes memory that merely lies between rows."""
import pytest
import torch

from paged_mla_speculative_gb300 import binding as mb
from tests.test_evict_gpu import Case, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def arguments(case):
    """Every array of 32-bit words in a block of one tensor of its own."""
    n, width = len(case.lens), case.weights.shape[1]
    stack = case.stack + [-1] * (case.units - len(case.stack))
    arrays = dict(kv_indices=case.indices, kv_indptr=case.indptr, kv_lens=case.lens, page_refs=case.refs, free_pages=stack,
                  free_count=[len(case.stack)], new_indices=[-9] * (-(-600 // case.page)), new_indptr=[-9] * (n + 1), new_lens=[-9] * n)
    args = {k: _i32(v) for k, v in arrays.items()}
    return dict(args, weights=case.weights, budget=100, kv_cache=case.cache, new_weights=torch.full((n, width), -9.0, device="cuda"))


@pytest.mark.parametrize("page", [1, 64])
def test_overlaps_are_refused(page):
    case = Case([200, 300, 120, 150], page, 1600 // page + 40, layers=2, seed=1)
    with case.plan() as plan:
        args = arguments(case)
        before = {k: v.clone() for k, v in args.items() if isinstance(v, torch.Tensor)}

        def refused(**bad):
            with pytest.raises(mb.MlaVerifyError) as e:
                mb.evict_kv(plan, **dict(args, **bad))
            assert e.value.status == -9

        words = torch.zeros(60000, dtype=torch.int32, device="cuda")
        tables = ("new_indices", "new_indptr", "new_lens", "page_refs", "free_pages", "free_count")
        for out in tables:
            for other in tables + ("kv_indices", "kv_indptr", "kv_lens"):
                if other == out:
                    continue
                # `out` begins at `other`'s last words, then ends at its first ones.
                n, m = args[out].numel(), args[other].numel()
                for at in ((m - 1) // 4 * 4, -((n - 1) // 4 * 4)):
                    base = max(0, -at)
                    refused(**{other: words[base:base + m], out: words[base + at:base + at + n]})
        width = args["weights"].shape[1]
        floats = torch.zeros(4 * 2 * width, device="cuda")
        wide = floats.view(4, 2 * width)[:, :width]
        for out in ("new_indices", "new_indptr", "new_lens", "free_count"):
            for at in (0, 3 * 2 * width):   # in the first row and in the last
                inside = floats.view(torch.int32)[at:at + args[out].numel()]
                refused(weights=wide, **{out: inside})
                refused(new_weights=wide, **{out: inside})
        if page == 64:
            cache = case.cache.contiguous().view(torch.int32).flatten()
            for at in (0, cache.numel() - 4):
                refused(kv_cache=cache.view(torch.bfloat16).view(2, -1, 576), new_lens=cache[at:at + 4])
        refused(new_weights=args["weights"])
        refused(weights=floats[:4 * width].view(4, width), new_weights=floats[4:4 + 4 * width].view(4, width))
        torch.cuda.synchronize()
        assert plan.get_error() == 0
        for k, v in before.items():
            assert torch.equal(args[k].view(torch.int16), v.view(torch.int16)), k


@pytest.mark.parametrize("page", [1, 64])
def test_rows_side_by_side(page):
    """Weights and new weights as [requests, 2, width], the new tables behind the
    rows of a wide array: nothing overlaps, and the results are those of arrays apart."""
    results = []
    for beside in (False, True):
        case = Case([200, 300, 120, 150], page, 1600 // page + 40, layers=2, seed=2)
        with case.plan() as plan:
            args = arguments(case)
            width = args["weights"].shape[1]
            if beside:
                both = torch.full((4, 3, width + 4 - width % 4), -9.0, device="cuda")
                both[:, 0, :width] = args["weights"]
                args.update(weights=both[:, 0, :width], new_weights=both[:, 1, :width], new_indptr=both[0, 2].view(torch.int32)[:5],
                            new_lens=both[1, 2].view(torch.int32)[:4])
                if page == 64:
                    layers = torch.zeros(2, case.cache.shape[1] + 64, 576, dtype=torch.bfloat16, device="cuda")
                    layers[:, :-64] = case.cache
                    args.update(kv_cache=layers[:, :-64], new_indices=layers[0, -64:].view(torch.int32).flatten()[:10])
            got = mb.evict_kv(plan, **args, sink=4, recent=20, extra_rows=3)
            torch.cuda.synchronize()
            assert plan.get_error() == 0
            total = int(got[1][-1])
            results.append([got[0][:total].tolist(), got[1].tolist(), got[2].tolist(), got[3].contiguous().view(torch.int32),
                            *(args[k] for k in ("page_refs", "free_pages", "free_count")),
                            *([args["kv_cache"].contiguous().view(torch.int32)] if page == 64 else [])])
    for a, b in zip(*results):
        assert torch.equal(a, b) if isinstance(a, torch.Tensor) else a == b
