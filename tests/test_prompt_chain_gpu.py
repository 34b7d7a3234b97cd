"""A long append_kv followed at once by the attention that reads its queries and
rows, and by another append_kv that reads what the first wrote: the kernels
overlap their launches, and no byte may be read before it is written."""
import pytest
import torch

from paged_mla_speculative_gb300 import binding as mb

pytestmark = pytest.mark.gpu

N, H, B, T, P = 8192, 64, 8, 8, 1000      # the last B * T tokens are the drafts; the first P are shared


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_mla_speculative_gb300 import build
    build.build()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_attention_right_behind_a_long_append():
    g = torch.Generator(device="cuda").manual_seed(7)
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)  # noqa: E731
    t = torch.arange(N, device="cuda", dtype=torch.float64)
    angle = t[:, None] * 10000.0 ** (-torch.arange(0, 64, 2, device="cuda", dtype=torch.float64) / 64)
    cos_sin = torch.cat((angle.cos(), angle.sin()), -1).float()
    weight = bf(512)
    slots = torch.randperm(N, generator=g, device="cuda").int()
    position = torch.arange(N, device="cuda").int()
    first = N - B * T
    idx = torch.cat([torch.cat((slots[:P], slots[first + b * T:first + (b + 1) * T])) for b in range(B)]).contiguous()
    ptr, lens = _i32([b * (P + T) for b in range(B + 1)]), _i32([P + T] * B)
    parent, groups, shared = _i32([list(range(-1, T - 1))] * B), _i32([0, B]), _i32([P])
    data = [(bf(N, 576), bf(N, H, 512), bf(N, H, 64)) for _ in range(3)]
    with mb.Plan(B, T, H, 1, N, P + T) as plan:
        def step(kv, nope, pe, cache, q, again, wait):
            mb.append_kv(plan, kv, weight, 1e-6, cos_sin, position, slots, cache, q_nope=nope, q_pe=pe, q=q)
            wait()
            out, lse = mb.mla_verify_attn_shared(plan, q[first:].view(B, T, H, 576), cache, idx, ptr, lens, parent, 0.07, groups,
                                                 shared)
            wait()
            mb.append_kv(plan, kv, weight, 1e-6, cos_sin, position, slots, cache, q_nope=nope, q_pe=pe, q=q)
            wait()
            # the queries just written, copied and rotated once more
            mb.append_kv(plan, kv, weight, 1e-6, cos_sin, position, slots, cache, q_nope=q[..., :512], q_pe=q[..., 512:], q=again)
            wait()
            return out, lse
        room = lambda: (torch.zeros(N, 576, dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                        torch.zeros(N, H, 576, dtype=torch.bfloat16, device="cuda"),
                        torch.zeros(N, H, 576, dtype=torch.bfloat16, device="cuda"))
        behind, alone = room(), room()
        for x in data * 3:          # every pass finds the last one's queries and rows in the buffers
            torch.cuda.synchronize()
            got = step(*x, *behind, lambda: None)
            torch.cuda.synchronize()
            want = step(*x, *alone, torch.cuda.synchronize)
            for a, b in zip(got + behind, want + alone):
                assert torch.equal(a, b)
        assert plan.get_error() == 0
