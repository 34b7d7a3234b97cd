"""Forking and freeing requests of a counted page pool on the GPU: tables,
counts, the stack of free pages, every row of every layer and the status bits
equal the oracle's exactly."""
import random

import pytest
import torch

import oracle.page_pool_ref as pp
from paged_mla_speculative_gb300 import binding as mb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def _i32(v):
    return torch.tensor(list(v) if len(v) else [0], dtype=torch.int32)[:len(v)].cuda()


class Pool:
    """The device arrays of a pool and, beside them, the oracle's lists."""

    def __init__(self, pages, layers=1, seed=0, pad=0):
        self.rng = random.Random(seed)
        self.pages, self.layers = pages, layers
        g = torch.Generator().manual_seed(seed)
        # a row is told by its number; layers may lie further apart than one cache
        rows = torch.randperm(layers * (pages * 64 + pad), generator=g).reshape(layers, pages * 64 + pad)
        store = rows.reshape(layers, -1, 1).expand(-1, -1, 288).int().contiguous()
        self.cache = store.view(torch.bfloat16).cuda()[:, :pages * 64]
        self.rows = [r[:pages * 64].tolist() for r in rows]
        self.refs = [0] * pages
        self.stack = list(range(pages))
        self.rng.shuffle(self.stack)
        self.d_refs, self.d_count = _i32(self.refs), _i32([pages])
        self.d_free = _i32(self.stack)

    def request(self, n):
        table = [self.stack.pop() for _ in range(-(-n // 64))]
        for p in table:
            self.refs[p] = 1
        return table

    def push(self):
        """The oracle's state to the device."""
        self.d_refs.copy_(torch.tensor(self.refs))
        self.d_count.fill_(len(self.stack))
        self.d_free.fill_(-1)
        self.d_free[:len(self.stack)] = _i32(self.stack)

    def check(self):
        assert self.d_refs.tolist() == self.refs
        assert self.d_free[:int(self.d_count)].tolist() == self.stack
        got = self.cache.contiguous().view(torch.int32)
        assert (got == got[..., :1]).all()
        assert got[..., 0].tolist() == self.rows


def _tables(tables):
    ptr = [0]
    for t in tables:
        ptr.append(ptr[-1] + len(t))
    return [p for t in tables for p in t], ptr


def _fork(plan, pool, parents, tables, lens, extra=0, capacity=None, idx=None, ptr=None):
    i, p = _tables(tables)
    idx, ptr = idx or i, ptr or p
    pool.push()
    plan.get_error()
    room = sum(-(-(max(n, 0) + extra) // 64) for n in lens) * len(parents) + 4 if capacity is None else capacity
    out = torch.full((room + 4,), -9, dtype=torch.int32, device="cuda")
    ci, cp, cl = mb.fork_kv(plan, _i32(parents), _i32(idx), _i32(ptr), _i32(lens),
                            pool.cache if pool.layers > 1 else pool.cache[0], pool.d_refs, pool.d_free, pool.d_count,
                            extra_rows=extra, child_indices=out[:room])
    torch.cuda.synchronize()
    want, wl, pool.refs, pool.stack, flags = pp.fork_kv(parents, idx, ptr, lens, pool.rows, pool.refs, pool.stack, extra, room,
                                                        plan.max_kv_len)
    wi, wp = _tables(want)
    assert cp.tolist() == wp and cl.tolist() == wl
    assert out.tolist() == wi + [-9] * (room + 4 - len(wi))
    assert plan.get_error() == flags
    pool.check()
    return want, wl, flags


def _free(plan, pool, tables):
    pool.push()
    i, p = _tables(tables)
    mb.free_kv(plan, _i32(i or [0]), _i32(p), pool.d_refs, pool.d_free, pool.d_count)
    torch.cuda.synchronize()
    pool.refs, pool.stack, flags = pp.free_kv(tables, pool.refs, pool.stack)
    assert plan.get_error() == flags
    pool.check()
    return flags


def _plan(pool, max_len=4096, batch=1100):
    return mb.Plan(batch, 1, 1, 64, pool.pages * 64, max_len)


@pytest.mark.parametrize("layers,pad", [(1, 0), (3, 0), (2, 192)])
@pytest.mark.parametrize("lens", [[1], [64], [63, 65], [0, 300, 128, 1000]])
def test_fork_then_free_matches_the_oracle(lens, layers, pad):
    pool = Pool(96, layers, seed=len(lens), pad=pad)
    tables = [pool.request(n) for n in lens]
    with _plan(pool, batch=16) as plan:
        parents = [p for p in range(len(lens)) for _ in range(3)][::-1]
        for extra in (0, 1, 70):
            kids, kl, flags = _fork(plan, pool, parents, tables, lens, extra)
            assert flags == 0
            again, _, flags = _fork(plan, pool, [0, len(kids) - 1, 0], kids, kl, 0)   # children of children
            assert flags == 0
            assert _free(plan, pool, kids + again) == 0
        assert _free(plan, pool, tables) == 0
        assert len(pool.stack) == pool.pages and not any(pool.refs)


def test_more_children_than_threads():
    pool = Pool(1200, seed=4)
    lens = [70, 64, 1]
    tables = [pool.request(n) for n in lens]
    with _plan(pool) as plan:
        parents = [i % 3 for i in range(1100)]
        kids, _, flags = _fork(plan, pool, parents, tables, lens, 0)
        assert flags == 0
        assert _free(plan, pool, kids) == 0


def test_what_does_not_fit_is_cut_and_reported():
    pool = Pool(12, seed=6)
    lens = [100, 128, 300]
    tables = [pool.request(n) for n in lens]            # 2 + 2 + 5 pages: three are left
    with _plan(pool) as plan:
        kids, _, flags = _fork(plan, pool, [0, 0, 1, 2, 2, 1], tables, lens)
        assert flags == mb.DEV_CAPACITY and [len(k) for k in kids] == [2, 2, 2, 5, 0, 0]
        assert _free(plan, pool, kids) == 0
        kids, _, flags = _fork(plan, pool, [0, 1, 2], tables, lens, capacity=4)
        assert flags == mb.DEV_CAPACITY and [len(k) for k in kids] == [2, 2, 0]
        _free(plan, pool, kids)


def test_a_stack_height_that_cannot_be():
    pool = Pool(16, seed=16)
    lens = [100, 64]
    tables = [pool.request(n) for n in lens]
    i, p = _tables(tables)
    with _plan(pool) as plan:
        for height in (-1, 17):
            pool.push()
            pool.d_count.fill_(height)
            _, cp, cl = mb.fork_kv(plan, _i32([1, 0]), _i32(i), _i32(p), _i32(lens), pool.cache[0], pool.d_refs, pool.d_free,
                                   pool.d_count)
            # the child of full pages needs none of the stack
            assert plan.get_error() == mb.DEV_CAPACITY and int(pool.d_count) == height
            assert cp.tolist() == [0, 1, 1] and cl.tolist() == [64, 0]


def test_bad_parents_lengths_tables_and_pages():
    pool = Pool(64, 2, seed=7)
    lens = [100, 200, 64, 90]
    tables = [pool.request(n) for n in lens]
    with _plan(pool, max_len=256) as plan:
        _, _, flags = _fork(plan, pool, [0, 4, -1, 1], tables, lens)
        assert flags == mb.DEV_BAD_POOL
        _, _, flags = _fork(plan, pool, [0, 1, 2], tables, [100, -5, 64, 90], 10)
        assert flags == mb.DEV_BAD_LEN
        _, _, flags = _fork(plan, pool, [0, 1, 2], tables, lens, 60)
        assert flags == mb.DEV_BAD_LEN                    # 200 + 60 > 256
        _, _, flags = _fork(plan, pool, [0, 1, 2], tables, [100, 257, 64, 90])
        assert flags == mb.DEV_BAD_LEN
        _, _, flags = _fork(plan, pool, [0, 1], tables, [100, 200, 65, 129])
        assert flags == 0                                 # nobody forks the two wrong ones
        _, _, flags = _fork(plan, pool, [2, 3], tables, [100, 200, 65, 129])
        assert flags == mb.DEV_BAD_INDPTR
        broken = [list(t) for t in tables]
        broken[1][0], broken[1][3] = 64, -2               # a full page and the partial one
        _, _, flags = _fork(plan, pool, [1, 0], broken, lens)
        assert flags == mb.DEV_BAD_SLOT
        pool.refs[tables[3][0]] = 0                       # held, but not counted
        _, _, flags = _fork(plan, pool, [3], tables, lens)
        assert flags == mb.DEV_BAD_REF
        pool.stack[-1] = 64                               # the stack holds a page outside the cache
        _, _, flags = _fork(plan, pool, [0], tables, lens)
        assert flags == mb.DEV_BAD_SLOT
        pool.stack[-1] = tables[2][0]                     # ... and one that is in use
        _, _, flags = _fork(plan, pool, [0], tables, lens)
        assert flags == mb.DEV_BAD_REF


def test_freed_twice_and_pages_outside():
    pool = Pool(40, seed=8)
    lens = [100, 500]
    tables = [pool.request(n) for n in lens]
    with _plan(pool) as plan:
        assert _free(plan, pool, [tables[0], tables[0]]) == mb.DEV_BAD_REF
        assert _free(plan, pool, [tables[0]]) == mb.DEV_BAD_REF
        assert _free(plan, pool, [[40, -1], tables[1][:3], [], tables[1][3:]]) == mb.DEV_BAD_SLOT
        # a table that is none, or a stack that cannot be: nothing changes
        refs, stack = list(pool.refs), list(pool.stack)
        for ptr, bit in (([0, 2, 1, 3], mb.DEV_BAD_INDPTR), ([-1, 2, 3], mb.DEV_BAD_INDPTR)):
            mb.free_kv(plan, _i32(tables[1]), _i32(ptr), pool.d_refs, pool.d_free, pool.d_count)
            assert plan.get_error() == bit
        for n in (-1, 41):
            pool.d_count.fill_(n)
            mb.free_kv(plan, _i32(tables[1]), _i32([0, 3]), pool.d_refs, pool.d_free, pool.d_count)
            assert plan.get_error() == mb.DEV_CAPACITY and int(pool.d_count) == n
        assert pool.d_refs.tolist() == refs


def test_large_pool_and_shared_pages():
    """Enough pages for several words per thread of the free's bit map, tables
    that share most of their pages, in one call; twice, with the same result."""
    pool = Pool(300_000, seed=9)
    pool.cache, pool.rows = torch.zeros(1, 64, 576, dtype=torch.bfloat16, device="cuda"), []
    tables = [pool.request(64 * 700) for _ in range(40)]
    for t in tables[1:]:
        for j in range(0, 700, 2):                       # every second page is the first table's
            pool.refs[t[j]] = 0
            t[j] = tables[0][j]
            pool.refs[t[j]] += 1
    start = list(pool.refs), list(pool.stack)
    with mb.Plan(40, 1, 1, 64, 300_000 * 64, 64) as plan:
        seen = []
        for _ in range(2):
            pool.refs, pool.stack = list(start[0]), list(start[1])
            pool.push()
            i, p = _tables(tables)
            mb.free_kv(plan, _i32(i), _i32(p), pool.d_refs, pool.d_free, pool.d_count)
            torch.cuda.synchronize()
            pool.refs, pool.stack, flags = pp.free_kv(tables, pool.refs, pool.stack)
            assert plan.get_error() == flags == 0
            assert pool.d_refs.tolist() == pool.refs
            seen.append(pool.d_free[:int(pool.d_count)].tolist())
            assert seen[-1] == pool.stack
        assert seen[0] == seen[1]


def test_captured_beam_steps_on_another_stream():
    """Fork and free captured into one graph, replayed: each replay continues
    from the device's own stack and counts."""
    pool = Pool(64, 2, seed=10)
    lens = [130, 64, 70]
    tables = [pool.request(n) for n in lens]
    pool.push()
    with _plan(pool, batch=4) as plan:
        i, p = _tables(tables)
        di, dp, dl, par = _i32(i), _i32(p), _i32(lens), _i32([2, 0, 0, 1])
        ci, cp, cl = _i32([0] * 16), _i32([0] * 5), _i32([0] * 4)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            mb.fork_kv(plan, par, di, dp, dl, pool.cache, pool.d_refs, pool.d_free, pool.d_count, 5, ci, cp, cl, stream=s)
            mb.free_kv(plan, ci, cp, pool.d_refs, pool.d_free, pool.d_count, stream=s)
        for _ in range(3):
            g.replay()
            torch.cuda.synchronize()
            kids, kl, pool.refs, pool.stack, f0 = pp.fork_kv([2, 0, 0, 1], i, p, lens, pool.rows, pool.refs, pool.stack, 5, 16,
                                                             4096)
            pool.refs, pool.stack, f1 = pp.free_kv(kids, pool.refs, pool.stack)
            assert f0 == f1 == plan.get_error() == 0
            assert cp.tolist() == _tables(kids)[1] and ci.tolist()[:int(cp[-1])] == _tables(kids)[0] and cl.tolist() == kl
            pool.check()


def test_host_argument_errors():
    pool = Pool(8)
    t = pool.request(100)
    pool.push()
    a = [_i32([0]), _i32(t), _i32([0, 2]), _i32([100])]
    out = [_i32([0] * 8), _i32([0, 0]), _i32([0])]
    lib = mb.load_library()
    with mb.Plan(2, 1, 1, 64, 512, 256) as plan, mb.Plan(2, 1, 1, 1, 512, 256) as flat:
        def fork(plan=plan, c=1, p=1, layers=1, stride=0, extra=0, cap=8, **null):
            ptr = dict(par=a[0], idx=a[1], indptr=a[2], lens=a[3], cache=pool.cache, refs=pool.d_refs, free=pool.d_free,
                       count=pool.d_count, ci=out[0], cp=out[1], cl=out[2])
            x = {k: null[k] if k in null else v.data_ptr() for k, v in ptr.items()}
            return lib.mla_verify_fork_kv(plan.handle, c, x["par"], p, x["idx"], x["indptr"], x["lens"], x["cache"], layers,
                                          stride, extra, x["refs"], x["free"], x["count"], x["ci"], cap, x["cp"], x["cl"], None)

        def free(plan=plan, b=1, **null):
            ptr = dict(idx=a[1], indptr=a[2], refs=pool.d_refs, free=pool.d_free, count=pool.d_count)
            x = {k: null[k] if k in null else v.data_ptr() for k, v in ptr.items()}
            return lib.mla_verify_free_kv(plan.handle, b, x["idx"], x["indptr"], x["refs"], x["free"], x["count"], None)
        for k in ("par", "idx", "indptr", "lens", "cache", "refs", "free", "count", "ci", "cp", "cl"):
            assert fork(**{k: None}) == -1 and fork(**{k: pool.d_refs.data_ptr() + 4}) == -2, k
        for k in ("idx", "indptr", "refs", "free", "count"):
            assert free(**{k: None}) == -1 and free(**{k: pool.d_refs.data_ptr() + 4}) == -2, k
        assert fork(plan=flat) == -3 and free(plan=flat) == -3
        for c in (0, 3):
            assert fork(c=c) == -4 and fork(p=c) == -4 and free(b=c) == -4
        for bad in (dict(layers=0), dict(stride=-8), dict(stride=4), dict(extra=-1), dict(extra=257), dict(cap=-1)):
            assert fork(**bad) == -9, bad
        torch.cuda.synchronize()
        assert plan.get_error() == 0
        pool.check()
        assert fork() == 0 and free() == 0
        torch.cuda.synchronize()
        assert plan.get_error() == 0
