"""A serving step over shared prompts, as a program runs it: prompt rows
written (append_kv), requests forked, their drafts' rows and queries made, the
shared verify attention, and the requests freed -- eagerly, and as one captured
graph replayed with other tokens.  Each stage is checked against its oracle on
the bits that the stage before left."""
import numpy as np
import pytest
import torch

import oracle
import oracle.append_ref as ar
import oracle.page_pool_ref as pp
from paged_mla_speculative_gb300 import binding as mb
from tests import gpu_util as G
from tests.conftest import bits

pytestmark = pytest.mark.gpu

T, H, PAGES, SCALE = 4, 16, 64, 192 ** -0.5
LENS, CHILDREN = [150, 70], [0, 0, 0, 1, 1]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _bf16(x):
    """fp64 -> what one rounding to bf16 may give: (nearest, tolerance)."""
    return x, (2.0 ** -8 + 2.0 ** -16) * np.abs(x) + 2.0 ** -20


@pytest.mark.parametrize("captured", [False, True])
def test_prompt_fork_verify_free(captured):
    g = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    pos = torch.arange(512, dtype=torch.float64)
    angle = pos[:, None] * 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    cos_sin = torch.cat((angle.cos(), angle.sin()), -1).float().cuda()
    weight = (1 + 0.2 * torch.randn(512, generator=g)).to(torch.bfloat16).cuda()
    cache = torch.zeros(PAGES * 64, 576, dtype=torch.bfloat16, device="cuda")
    stack = list(np.random.default_rng(4).permutation(PAGES))
    tables = [[int(stack.pop()) for _ in range(-(-n // 64))] for n in LENS]
    refs = [0] * PAGES
    for p in sum(tables, []):
        refs[p] = 1
    d_refs, d_count = _i32(refs), _i32([len(stack)])
    d_free = _i32([int(x) for x in stack] + [-1] * (PAGES - len(stack)))
    idx, ptr = _i32(sum(tables, [])), _i32([0, len(tables[0]), sum(map(len, tables))])
    B = len(CHILDREN)
    with mb.Plan(B, T, H, 64, PAGES * 64, 256) as plan:
        # The prompts' rows, in one call.
        N = sum(LENS)
        kv = rand(N, 576)
        where = [(r, j) for r, n in enumerate(LENS) for j in range(n)]
        slots = [tables[r][j // 64] * 64 + j % 64 for r, j in where]
        mb.append_kv(plan, kv.cuda(), weight, 1e-6, cos_sin, _i32([j for _, j in where]), _i32(slots), cache)
        torch.cuda.synchronize()
        w64, cs64 = weight.double().cpu().numpy(), cos_sin.double().cpu().numpy()
        none = np.zeros((N, 0, 64))
        ref, _, _ = ar.append_kv(kv.double().numpy(), w64, 1e-6, None, none, cs64, [j for _, j in where], slots, False,
                                 np.zeros((PAGES * 64, 576)), np.zeros((N, 0, 576)))
        near, tol = _bf16(ref)
        assert (np.abs(cache.double().cpu().numpy() - near) <= tol).all()

        # One verify step: its inputs, and the program that runs it.
        parents, group_indptr = _i32(CHILDREN), _i32([0, 3, 5])
        shared = _i32([n // 64 * 64 for n in LENS])
        d_lens = _i32(LENS)
        draft_kv = torch.zeros(B * T, 576, dtype=torch.bfloat16, device="cuda")
        q_nope = torch.zeros(B * T, H, 512, dtype=torch.bfloat16, device="cuda")
        q_pe = torch.zeros(B * T, H, 64, dtype=torch.bfloat16, device="cuda")
        parent = _i32([[-1, 0, 0, 2]] * B)
        ci, cp, cl = _i32([0] * 32), _i32([0] * (B + 1)), _i32([0] * B)
        q = torch.zeros(B * T, H, 576, dtype=torch.bfloat16, device="cuda")
        out, lse = plan.new_outputs(B)
        depth = torch.tensor([0, 1, 1, 2], device="cuda").repeat(B)
        state = {}

        def step():
            mb.fork_kv(plan, parents, idx, ptr, d_lens, cache, d_refs, d_free, d_count, T, ci, cp, cl)
            j = (cl[:, None] - T + torch.arange(T, device="cuda")).flatten()          # logical rows of the drafts
            slot = ci[cp[:-1].repeat_interleave(T, output_size=B * T) + j // 64] * 64 + j % 64
            position = (cl - T).repeat_interleave(T, output_size=B * T) + depth
            state["slot"], state["position"] = slot.int(), position.int()
            mb.append_kv(plan, draft_kv, weight, 1e-6, cos_sin, state["position"], state["slot"], cache, q_nope=q_nope,
                         q_pe=q_pe, q=q)
            mb.mla_verify_attn_shared(plan, q.view(B, T, H, 576), cache, ci, cp, cl, parent, SCALE, group_indptr, shared, out, lse)
            mb.free_kv(plan, ci, cp, d_refs, d_free, d_count)

        run = step
        if captured:
            warm = torch.cuda.Stream()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=warm):
                step()
            run = graph.replay
        o_refs, o_stack = list(refs), [int(x) for x in stack]
        for _ in range(3):
            new = rand(B * T, 576), rand(B * T, H, 512), rand(B * T, H, 64)
            for d, v in zip((draft_kv, q_nope, q_pe), new):
                d.copy_(v)
            before = cache.double().cpu().numpy()
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            assert plan.get_error() == 0
            rows = list(before)
            want, wl, o_refs, o_stack, f = pp.fork_kv(CHILDREN, sum(tables, []), [0, len(tables[0]), sum(map(len, tables))], LENS,
                                                      [rows], o_refs, o_stack, T, 32, 256)
            assert f == 0 and cl.tolist() == wl and ci[:int(cp[-1])].tolist() == sum(want, [])
            slots = [want[b][(wl[b] - T + t) // 64] * 64 + (wl[b] - T + t) % 64 for b in range(B) for t in range(T)]
            assert state["slot"].tolist() == slots
            ref, ref_q, f = ar.append_kv(new[0].double().numpy(), w64, 1e-6, new[1].double().numpy(), new[2].double().numpy(), cs64,
                                         state["position"].tolist(), slots, False, np.array(rows), np.zeros((B * T, H, 576)))
            assert f == 0
            for got, x in ((cache, ref), (q, ref_q)):
                near, tol = _bf16(x)
                assert (np.abs(got.double().cpu().numpy() - near) <= tol).all()
            ro, rl = oracle.mla_verify(bits(q.view(B, T, H, 576)), bits(cache), np.array(sum(want, [])), cp.cpu().numpy(),
                                       np.array(wl), parent.cpu().numpy(), SCALE, 64)
            G.assert_parity(out.cpu().numpy(), lse.cpu().numpy(), ro, rl)
            o_refs, o_stack, f = pp.free_kv(want, o_refs, o_stack)
            assert f == 0 and d_refs.tolist() == o_refs == refs and d_free[:int(d_count)].tolist() == o_stack
