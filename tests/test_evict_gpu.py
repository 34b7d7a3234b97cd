"""Eviction on the GPU: tables, weights, counts, the stack of free pages, every
row of every layer and the status bits equal the oracle's exactly."""
import random

import pytest
import torch

from oracle import evict_ref as E
from paged_mla_speculative_gb300 import binding as mb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def _i32(v):
    return torch.tensor(list(v) if len(v) else [0], dtype=torch.int32).cuda()


class Case:
    """Requests of a pool (lists, and the device's copies of them)."""

    def __init__(self, lens, page, units, layers=1, seed=0, values="mixed", pad=0, width=None, max_len=None):
        rng = self.rng = random.Random(seed)
        self.page, self.units, self.layers = page, units, layers
        ids = list(range(units))
        rng.shuffle(ids)
        self.lens, self.indices, self.indptr = list(lens), [], [0]
        for n in lens:
            self.indices += [ids.pop() for _ in range(-(-n // page))]
            self.indptr.append(len(self.indices))
        self.refs = [0] * units
        for u in self.indices:
            self.refs[u] = 1
        self.stack = ids
        g = torch.Generator().manual_seed(seed)
        self.max_len = max_len or max(max(lens), 1) + 100
        shape = (len(lens), width or self.max_len)
        w = torch.rand(shape, generator=g)
        if values == "ties":
            w = (w * 4).round() / 4
        elif values == "mixed":
            pick = torch.rand(shape, generator=g)
            w = torch.where(pick < 0.3, 0.0, w)
            for i, v in enumerate((-0.0, float("nan"), float("inf"), float("-inf"), -1.0, 1e-42, 1e38)):
                w[(pick > 0.9 + 0.01 * i) & (pick <= 0.91 + 0.01 * i)] = v
        elif values == "same":
            w[:] = 0.5
        elif values == "near":      # keys that differ in their lowest bits alone
            w = (torch.full(shape, 0x3f800000, dtype=torch.int32) + torch.randint(0, 40, shape, generator=g, dtype=torch.int32)).view(
                torch.float32)
        self.weights = w.cuda()
        self.rows = self.cache = None
        if page == 64:
            rows = torch.randperm(layers * (units * 64 + pad), generator=g).reshape(layers, units * 64 + pad)
            self.cache = rows.reshape(layers, -1, 1).expand(-1, -1, 288).int().contiguous().view(torch.bfloat16).cuda()[:, :units * 64]
            self.rows = [r[:units * 64].tolist() for r in rows]

    def plan(self, batch=None):
        return mb.Plan(batch or len(self.lens), 1, 1, self.page, self.units * self.page, self.max_len)

    def evict(self, plan, budget, sink=0, recent=0, extra=0, capacity=None, count=None, want=None):
        pool = [_i32(self.refs), torch.full((self.units,), -1, dtype=torch.int32).cuda(), _i32([len(self.stack)])]
        if self.stack:
            pool[1][:len(self.stack)] = _i32(self.stack)
        if count is not None:
            pool[2].fill_(count)
        room = capacity if capacity is not None else sum(-(-(min(max(n, 0), budget) + extra) // self.page) for n in self.lens) + 3
        out = torch.full((room + 8,), -9, dtype=torch.int32, device="cuda")
        ptr, lens = _i32([-9] * (len(self.lens) + 1)), _i32([-9] * len(self.lens))
        new = torch.full((len(self.lens), self.weights.shape[1] + 5), -9.0, device="cuda")
        plan.get_error()
        cache = None if self.cache is None else self.cache if self.layers > 1 else self.cache[0]
        got = mb.evict_kv(plan, self.weights, budget, _i32(self.indices), _i32(self.indptr), _i32(self.lens), cache, *pool, sink=sink,
                          recent=recent, extra_rows=extra, new_indices=out[:room], new_indptr=ptr, new_lens=lens, new_weights=new)
        torch.cuda.synchronize()
        assert got[0].data_ptr() == out.data_ptr() and got[3] is new
        if want is not None:
            return plan.get_error(), out, ptr, lens, new, pool
        ref = E.evict_kv([r.tolist() for r in self.weights.cpu()], budget, sink, recent, extra, self.page, self.indices, self.indptr,
                         self.lens, self.rows, self.refs, self.stack, room, plan.max_kv_len)
        tables, wl, ww, self.refs, self.stack, flags = ref
        assert lens.tolist() == wl
        wp = [0]
        for t in tables:
            wp.append(wp[-1] + len(t))
        assert ptr.tolist() == wp
        flat = [u for t in tables for u in t]
        assert out.tolist() == flat + [-9] * (room + 8 - len(flat))
        expect = torch.zeros_like(new, device="cpu")
        expect[:, :self.weights.shape[1]] = torch.tensor(ww)
        assert torch.equal(new.cpu().view(torch.int32), expect.view(torch.int32)) or (
            (new.cpu() == expect) | (new.cpu().isnan() & expect.isnan())).all()
        assert plan.get_error() == flags
        assert pool[0].tolist() == self.refs
        assert int(pool[2]) == len(self.stack) and pool[1][:len(self.stack)].tolist() == self.stack
        if self.cache is not None:
            rows = self.cache.contiguous().view(torch.int32)
            assert (rows == rows[..., :1]).all()
            assert rows[..., 0].tolist() == self.rows
        return flags, tables, wl, new


@pytest.mark.parametrize("page", [1, 64])
@pytest.mark.parametrize("values", ["mixed", "ties", "same", "near"])
@pytest.mark.parametrize("lens,budget,sink,recent,extra", [
    ([1], 0, 0, 0, 0),                              # nothing is kept
    ([5], 1, 0, 0, 1),
    ([64, 65, 128], 64, 0, 0, 0),
    ([300], 100, 70, 5, 8),                         # one page stays
    ([300, 0, 10, 130], 130, 4, 60, 0),             # within the budget, empty, equal to it
    ([200], 150, 100, 50, 1),                       # nothing to choose
    ([1000, 999, 3], 257, 128, 0, 70),
    ([700], 699, 0, 699, 0),                        # the first row alone goes
])
def test_matches_the_oracle(lens, budget, sink, recent, extra, values, page):
    units = sum(-(-n // page) + -(-(min(n, budget) + extra) // page) for n in lens) + 9
    case = Case(lens, page, units, layers=1 + len(lens) % 2, seed=sum(lens), values=values, pad=64 * (len(lens) % 2 == 0))
    with case.plan() as plan:
        assert case.evict(plan, budget, sink, recent, extra)[0] == 0


@pytest.mark.parametrize("page", [1, 64])
@pytest.mark.parametrize("n", [2048, 2049, 4097, 20000, 70000])
def test_long_requests(n, page):
    """One to eight CTAs a request."""
    for values in ("mixed", "ties"):
        case = Case([n, n // 3], page, 2 * n // page + 2000 // page + 40, seed=n, values=values, max_len=n + 1)
        with case.plan() as plan:
            assert case.evict(plan, n // 4, 5, 100, 1)[0] == 0


def test_more_rows_than_a_cta_holds():
    case = Case([250000], 1, 300000, seed=1, max_len=250000)
    with case.plan() as plan:
        assert case.evict(plan, 100000, 3, 7)[0] == 0


def test_a_batch_of_many_requests():
    lens = [i % 150 for i in range(1200)]
    for page in (1, 64):
        case = Case(lens, page, 200000 if page == 1 else 6000, seed=2, max_len=200)
        with case.plan() as plan:
            assert case.evict(plan, 66, 2, 10, 3)[0] == 0


def test_again_and_again():
    """Each call goes on with the tables and weights of the one before."""
    for page in (1, 64):
        case = Case([500, 320, 64], page, 3000 // page + 30, layers=2 if page == 64 else 1, seed=3, max_len=600)
        with case.plan() as plan:
            for budget in (400, 300, 299, 65, 3):
                flags, tables, lens, new = case.evict(plan, budget, 1, 2)
                assert flags == 0
                case.lens, case.indices, case.indptr = lens, [u for t in tables for u in t], [0]
                for t in tables:
                    case.indptr.append(case.indptr[-1] + len(t))
                case.weights = new[:, :case.max_len].contiguous()


def test_shared_entries_are_left_to_the_others():
    """Pages of two tables of the call, of tables outside it, twice in one."""
    for page in (1, 64):
        case = Case([300, 300, 129], page, 4000 // page + 20, seed=4)
        p = case.indptr
        share = 100 // page
        for i in range(share):
            case.refs[case.indices[p[1] + i]] = 0
            case.indices[p[1] + i] = case.indices[i]
            case.refs[case.indices[i]] = 2
        case.refs[case.indices[0]] += 3
        case.refs[case.indices[p[2]]] = 2
        case.indices[p[2] + 1] = case.indices[p[2]]
        with case.plan() as plan:
            assert case.evict(plan, 70, 0, 1)[0] == 0


def test_entries_behind_the_rows_are_given_back():
    for page in (1, 64):
        case = Case([300, 64], page, 2000 // page + 20, seed=5)
        case.lens = [100, 40]
        with case.plan() as plan:
            assert case.evict(plan, 90, 0, 0, 2)[0] == 0


@pytest.mark.parametrize("page", [1, 64])
def test_what_does_not_fit_is_cut_and_reported(page):
    def make():
        return Case([200, 300, 10, 100], page, sum(-(-n // page) for n in (200, 300, 10, 100)) + 128 // page * 2, seed=6)
    entries = -(-100 // page)
    for capacity in (1, entries, 2 * entries, 2 * entries + (page == 1)):
        case = make()
        with case.plan() as plan:
            assert case.evict(plan, 100, capacity=capacity)[0] == mb.DEV_CAPACITY
    case = make()                                      # the stack runs out
    case.stack = case.stack[:3]
    with case.plan() as plan:
        assert case.evict(plan, 100, extra=2 if page == 1 else 0)[0] == mb.DEV_CAPACITY


@pytest.mark.parametrize("page", [1, 64])
def test_requests_that_are_out_of_order(page):
    for name, at, value, flag in (("lens", 1, -1, mb.DEV_BAD_LEN), ("lens", 1, 9999, mb.DEV_BAD_LEN),
                                  ("indptr", 2, 1, mb.DEV_BAD_INDPTR), ("indptr", 1, -4, mb.DEV_BAD_INDPTR)):
        case = Case([200, 300, 10], page, 1500 // page + 20, seed=7)
        getattr(case, name)[at] = value
        with case.plan() as plan:
            assert case.evict(plan, 100)[0] & flag
    case = Case([200, 300, 10], page, 1500 // page + 20, seed=7)      # no room for more rows in the plan
    with case.plan() as plan:
        assert case.evict(plan, 400, extra=150)[0] == mb.DEV_BAD_LEN


@pytest.mark.parametrize("page", [1, 64])
def test_entries_and_counts_that_are_out_of_order(page):
    case = Case([200, 300], page, 1200 // page + 20, seed=8)
    case.indices[0], case.indices[-1], case.indices[2] = -1, case.units, 1 << 30
    case.refs[case.indices[1]] = 0
    case.stack[-1], case.stack[0] = case.units + 5, 0
    case.refs[case.stack[-2]] = 7
    with case.plan() as plan:
        assert case.evict(plan, 70, 66, 0, 66)[0] & mb.DEV_BAD_SLOT
    for count in (-1, case.units + 1):
        case = Case([200, 300], page, 1200 // page + 20, seed=8)
        with case.plan() as plan:
            err, out, ptr, lens, new, pool = case.evict(plan, 70, count=count, want=True)
        assert err == mb.DEV_CAPACITY and ptr.tolist() == [0, 0, 0] and lens.tolist() == [0, 0] and (out == -9).all()
        assert int(pool[2]) == count and pool[0].tolist() == case.refs and (new == 0).all()


def test_nothing_marked_is_left_behind():
    """A call that serves nobody, then one that does, on one plan; then a free."""
    case = Case([200, 300], 64, 40, seed=9)
    with case.plan() as plan:
        assert case.evict(plan, 100, capacity=1)[0] == mb.DEV_CAPACITY
        flags, tables, _, _ = case.evict(plan, 100)
        assert flags == 0
        ptr = [0, len(tables[0]), len(tables[0]) + len(tables[1])]
        refs, free, count = _i32(case.refs), _i32(case.stack + [-1] * (40 - len(case.stack))), _i32([len(case.stack)])
        mb.free_kv(plan, _i32(tables[0] + tables[1]), _i32(ptr), refs, free, count)
        assert int(count) == 40 and not refs.any() and sorted(free.tolist()) == list(range(40))


def test_captured_and_replayed_and_default_outputs():
    case = Case([200, 300, 20], 64, 60, layers=2, seed=10)
    with case.plan() as plan:
        args = [case.weights, 100, _i32(case.indices), _i32(case.indptr), _i32(case.lens), case.cache.contiguous()]
        pools = [[_i32(case.refs), torch.cat((_i32(case.stack), _i32([-1] * (60 - len(case.stack))))), _i32([len(case.stack)])]
                 for _ in range(3)]
        eager = mb.evict_kv(plan, *args, *pools[0], sink=3, recent=9, extra_rows=4)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        other = mb.evict_kv(plan, *args, *pools[1], sink=3, recent=9, extra_rows=4, stream=side)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            third = mb.evict_kv(plan, *args, *pools[2], sink=3, recent=9, extra_rows=4)
        graph.replay()
        torch.cuda.synchronize()
        assert plan.get_error() == 0
    total = int(eager[1][-1])
    assert eager[0].numel() == 3 * 2
    for got in (other, third):
        assert torch.equal(got[0][:total], eager[0][:total])
        assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(got[1:], eager[1:]))
    for pool in pools[1:]:
        assert all(torch.equal(a, b) for a, b in zip(pool, pools[0]))


def test_refusals():
    case = Case([200, 300], 64, 40, layers=2, seed=11)
    with case.plan() as plan:
        w = case.weights
        args = dict(weights=w, budget=100, kv_indices=_i32(case.indices), kv_indptr=_i32(case.indptr), kv_lens=_i32(case.lens),
                    kv_cache=case.cache, page_refs=_i32(case.refs), free_pages=_i32([0] * 40), free_count=_i32([0]))
        for bad in (dict(weights=w.double()), dict(weights=w[:, :-1]), dict(weights=w[:1]), dict(page_refs=_i32([0] * 39)),
                    dict(free_count=_i32([0, 0])), dict(kv_lens=_i32(case.lens).long()), dict(kv_cache=case.cache[:, :64]),
                    dict(new_lens=_i32([0])), dict(new_indptr=_i32([0, 0])), dict(new_weights=torch.zeros(2, 5, device="cuda")),
                    dict(new_weights=torch.zeros(1, 400, device="cuda").expand(2, 400))):
            with pytest.raises((TypeError, ValueError)):
                mb.evict_kv(plan, **dict(args, **bad))
        for bad in (dict(budget=-1), dict(sink=-1), dict(recent=-1), dict(sink=60, recent=41), dict(extra_rows=-1),
                    dict(extra_rows=case.max_len + 1), dict(new_weights=w), dict(new_indices=args["kv_indices"]),
                    dict(new_lens=args["kv_lens"]), dict(new_indptr=args["kv_indptr"]), dict(kv_cache=None),
                    dict(kv_cache=case.cache[0].expand(2, 40 * 64, 576))):
            with pytest.raises(mb.MlaVerifyError):
                mb.evict_kv(plan, **dict(args, **bad))
        for bad in (dict(budget=1 << 32), dict(budget=(1 << 32) + 100), dict(sink=1 << 40), dict(extra_rows=1 << 33)):
            with pytest.raises(ValueError):
                mb.evict_kv(plan, **dict(args, **bad))
        torch.cuda.synchronize()
        assert plan.get_error() == 0 and args["page_refs"].tolist() == case.refs


# Protected rows enough that they are copied while the others are chosen.
@pytest.mark.parametrize("lens,budget,sink,recent,extra,layers,max_len", [
    ([300, 500, 130, 64], 120, 5, 70, 8, 40, None),       # 64 is within the budget
    ([300, 500, 131, 0], 131, 66, 65, 0, 40, None),       # nothing besides is kept; a page stays; one is equal to the budget
    ([700], 300, 0, 130, 1, 67, None),                    # no leading row, layers that do not divide
    ([400, 333], 200, 63, 100, 0, 64, 13000),             # a cluster of two CTAs per request
    ([333, 400], 250, 1, 200, 0, 300, None),              # more than are copied early: the first of them go with the others
])
def test_protected_rows_of_many_layers(lens, budget, sink, recent, extra, layers, max_len):
    units = sum(-(-n // 64) + -(-(min(n, budget) + extra) // 64) for n in lens) + 3
    case = Case(lens, 64, units, layers=layers, seed=sum(lens), max_len=max_len, pad=64)
    with case.plan() as plan:
        assert case.evict(plan, budget, sink, recent, extra)[0] == 0


def test_protected_rows_of_requests_that_are_not_served_or_have_bad_pages():
    def make():
        return Case([300, 500, 130], 64, 30, layers=50, seed=10)
    for capacity in (1, 2, 4, 5):
        case = make()
        with case.plan() as plan:
            assert case.evict(plan, 120, 5, 70, capacity=capacity)[0] == mb.DEV_CAPACITY
    case = make()
    case.stack = case.stack[:3]
    with case.plan() as plan:
        assert case.evict(plan, 120, 5, 70)[0] == mb.DEV_CAPACITY
    case = make()
    case.lens[1] = 9999
    with case.plan() as plan:
        assert case.evict(plan, 120, 5, 70)[0] & mb.DEV_BAD_LEN
    case = make()
    case.indices[0], case.indices[-1], case.stack[-1] = -1, case.units, case.units + 5
    with case.plan() as plan:
        assert case.evict(plan, 120, 5, 70)[0] & mb.DEV_BAD_SLOT
