"""A prompt in chunks on a cache that is kept to a budget, as a serving program
runs it: rows appended, chunk attention, weights added up, eviction in every
layer, then a verify step on what is left -- eagerly against the oracles, and as
one captured graph that is replayed."""
import numpy as np
import pytest
import torch

from oracle import chunk_ref, evict_ref
from paged_mla_speculative_gb300 import binding as mb
from tests import chunk_util as C

pytestmark = pytest.mark.gpu

B, H, T, L, PAGES, LONGEST = 2, 16, 4, 2, 40, 520
CHUNKS = [[150, 70], [130, 0], [100, 140]]            # new tokens of each request, call by call
BUDGET, SINK, RECENT = 200, 70, 40


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Run:
    """Buffers of the run and its calls; nothing is allocated or read back in them."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(5)
        n = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.plan = mb.Plan(B, T, H, 64, PAGES * 64, LONGEST, torch.float32)
        self.weight = n(512)
        angle = torch.rand(600, 32, generator=g, device="cuda") * 6
        self.cos_sin = torch.cat((angle.cos(), angle.sin()), 1)
        lens = [sum(c[b] for c in CHUNKS) for b in range(B)]
        self.lens = lens
        entries = [-(-x // 64) for x in lens]
        ids = torch.randperm(PAGES, generator=g, device="cuda").int()
        self.table, self.ptr = ids[:sum(entries)].clone(), _i32(C.starts(entries))
        refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        refs[self.table.long()] = 1
        free = torch.full((PAGES,), -1, dtype=torch.int32, device="cuda")
        free[:PAGES - sum(entries)] = ids[sum(entries):]
        self.pool0 = [refs, free, _i32([PAGES - sum(entries)])]
        self.pool = [x.clone() for x in self.pool0]
        self.cache = n(L, PAGES * 64, 576)
        self.steps = []
        done = [0] * B
        host = ids.tolist()
        for new in CHUNKS:
            N = sum(new)
            positions = [done[b] + i for b in range(B) for i in range(new[b])]
            slots = [host[C.starts(entries)[b] + (done[b] + i) // 64] * 64 + (done[b] + i) % 64 for b in range(B) for i in range(new[b])]
            done = [d + c for d, c in zip(done, new)]
            pages = [-(-d // 64) for d in done]
            table = [host[C.starts(entries)[b] + e] for b in range(B) for e in range(pages[b])]
            self.steps.append(dict(
                new=new, lens=list(done), positions=_i32(positions), slots=_i32(slots), kv_indices=_i32(table),
                kv_indptr=_i32(C.starts(pages)), kv_lens=_i32(done), q_indptr=_i32(C.starts(new)),
                layers=[dict(kv=n(N, 576), q_nope=n(N, H, 512), q_pe=n(N, H, 64), q=torch.zeros(N, H, 576, device="cuda").bfloat16(),
                             out=torch.zeros(N, H, 512, device="cuda"), lse=torch.zeros(N, H, device="cuda")) for _ in range(L)]))
        self.weights = torch.zeros(B, LONGEST, device="cuda")
        self.new = dict(new_indices=torch.zeros(B * 8, dtype=torch.int32, device="cuda"), new_indptr=_i32([0] * (B + 1)),
                        new_lens=_i32([0] * B), new_weights=torch.zeros(B, LONGEST, device="cuda"))
        self.draft_q = n(L, B, T, H, 576)
        self.parent = (torch.arange(T, dtype=torch.int32, device="cuda") - 1).repeat(B, 1)
        self.out = torch.zeros(L, B, T, H, 512, device="cuda")
        self.lse = torch.zeros(L, B, T, H, device="cuda")

    def __call__(self):
        p = self.plan
        for x, y in zip(self.pool, self.pool0):
            x.copy_(y)
        self.weights.zero_()
        for s in self.steps:
            for cache, y in zip(self.cache, s["layers"]):
                mb.append_kv(p, y["kv"], self.weight, 1e-6, self.cos_sin, s["positions"], s["slots"], cache, q_nope=y["q_nope"],
                             q_pe=y["q_pe"], q=y["q"])
                tables = (y["q"], cache, s["kv_indices"], s["kv_indptr"], s["kv_lens"], s["q_indptr"])
                mb.mla_verify_attn_chunk(p, *tables, C.SCALE, out=y["out"], lse=y["lse"])
                mb.weigh_kv(p, *tables, y["lse"], C.SCALE, self.weights)
        mb.evict_kv(p, self.weights, BUDGET, s["kv_indices"], s["kv_indptr"], s["kv_lens"], self.cache, *self.pool, sink=SINK,
                    recent=RECENT, extra_rows=T, **self.new)
        for l in range(L):
            mb.mla_verify_attn(p, self.draft_q[l], self.cache[l], self.new["new_indices"], self.new["new_indptr"], self.new["new_lens"],
                               self.parent, C.SCALE, out=self.out[l], lse=self.lse[l])


def _results(run):
    return [y[k].clone() for s in run.steps for y in s["layers"] for k in ("out", "lse")] + [
        x.clone() for x in (run.weights, *run.new.values(), *run.pool, run.out, run.lse)]


def test_the_run_against_the_oracles():
    run = Run()
    before = run.cache.clone()
    run()
    torch.cuda.synchronize()
    assert run.plan.get_error() == 0
    total = np.zeros((B, LONGEST))
    tol = np.zeros((B, LONGEST))
    rows = [[None] * B for _ in range(L)]                 # each request's cached rows before the eviction
    for s in run.steps:
        for l, y in enumerate(s["layers"]):
            d = dict(q=y["q"].cpu(), cache=before[l].cpu(), page=64, **{k: s[k].cpu() for k in ("kv_indices", "kv_indptr", "kv_lens", "q_indptr")})
            slots = s["slots"].long().cpu()
            before[l][slots.cuda()] = run_rows(run, l, s)
            d["cache"] = before[l].cpu()
            C.assert_close(d, y["out"], y["lse"])
            for b, t0, t1, n, at, ok in C.requests(d):
                rows[l][b] = C.gather(d, at, ok)
                if t1 == t0:
                    continue
                q, lse = d["q"][t0:t1].double().numpy(), y["lse"][t0:t1].double().cpu().numpy()
                x = C.SCALE * (q.reshape(-1, 576) @ rows[l][b].T)
                seen = np.repeat(np.arange(n)[None] <= (n - (t1 - t0) + np.arange(t1 - t0))[:, None], H, 0)
                e = np.where(seen, np.exp(np.where(seen, x, 0) - lse.reshape(-1, 1)), 0)
                total[b, :n] += e.sum(0)
                tol[b, :n] += 1e-4 * e.sum(0) + 1e-6
    got = run.weights.double().cpu().numpy()
    assert (np.abs(got - total) <= tol).all()
    # The eviction, from the weights as they are.
    s = run.steps[-1]
    pool = [x.cpu().tolist() for x in run.pool0]
    host = [[(l, i) for i in range(PAGES * 64)] for l in range(L)]

    class Row(tuple):
        def __rmul__(self, k):
            return self

    host = [[Row(x) for x in layer] for layer in host]
    tables, lens, w, refs, stack, flags = evict_ref.evict_kv(
        run.weights.cpu().tolist(), BUDGET, SINK, RECENT, T, 64, s["kv_indices"].tolist(), s["kv_indptr"].tolist(), s["kv_lens"].tolist(),
        host, pool[0], pool[1][:pool[2][0]], B * 8, LONGEST)
    assert flags == 0 and run.new["new_lens"].tolist() == lens == [BUDGET + T] * B
    ptr = run.new["new_indptr"].tolist()
    assert [run.new["new_indices"].tolist()[ptr[b]:ptr[b + 1]] for b in range(B)] == tables
    assert run.pool[0].tolist() == refs and run.pool[1].tolist()[:len(stack)] == stack and int(run.pool[2]) == len(stack)
    assert torch.equal(run.new["new_weights"].cpu(), torch.tensor(w))
    # The verify step over the kept rows and the drafts' (whatever their places hold).
    for l in range(L):
        for b in range(B):
            kept = evict_ref.keep(run.weights[b].tolist(), run.lens[b], BUDGET, SINK, RECENT)
            at = [tables[b][j // 64] * 64 + j % 64 for j in range(BUDGET + T)]
            keys = run.cache[l][torch.tensor(at).cuda()].double().cpu().numpy()
            assert (keys[:BUDGET] == rows[l][b][kept]).all()
            o, lse, mass, size = chunk_ref.chunk_attn(run.draft_q[l, b].double().cpu().numpy(), keys, C.SCALE)
            assert np.abs(run.out[l, b].double().cpu().numpy() - o).max() <= 1e-2
            assert np.abs(run.lse[l, b].double().cpu().numpy() - lse).max() <= 1e-3


def run_rows(run, l, s):
    """The rows of a step's tokens as the cache held them: appended rows are
    checked by their own tests, and pages that the eviction filled are others."""
    free = set(run.pool0[1].tolist())
    slots = s["slots"].long()
    assert not {int(x) // 64 for x in slots} & free
    return run.cache[l][slots]


def test_captured_once_and_replayed():
    run = Run()
    start = run.cache.clone()
    run()
    torch.cuda.synchronize()
    eager = _results(run)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(2):
        run.cache.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        assert run.plan.get_error() == 0
        assert all(torch.equal(a, b) for a, b in zip(_results(run), eager))
