"""Inputs and bounds shared by the tests of chunks of new tokens and of weighed
rows (not a test module)."""
import numpy as np
import torch

from oracle import chunk_ref
from paged_mla_speculative_gb300 import binding as mb

SCALE = 192.0 ** -0.5


def starts(counts):
    return [0] + [int(x) for x in np.cumsum(counts)]


def make(new, lens, H, page=1, seed=0, front=0, pad=0, spike=0.01):
    """CPU inputs: request b has lens[b] rows, the last new[b] of them its new
    tokens'; `front` and `pad` tokens stand before and behind all of them."""
    g = torch.Generator().manual_seed(seed)
    entries = [-(-n // page) for n in lens]
    units = sum(entries) + 5
    if page == 1:
        units = -(-units // 64) * 64
    cache = torch.randn(units * page, 576, generator=g)
    cache[torch.rand(units * page, generator=g) < spike] *= 8
    N = front + sum(new) + pad
    q = torch.randn(N, H, 576, generator=g)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return dict(q=q.bfloat16(), cache=cache.bfloat16(), kv_indices=torch.randperm(units, generator=g)[:max(1, sum(entries))].int(),
                kv_indptr=i32(starts(entries)), kv_lens=i32(lens), q_indptr=i32([front + x for x in starts(new)]), page=page, H=H)


def plan_for(d, out_dtype=torch.float32, max_batch=None, max_kv_len=None, T=1):
    return mb.Plan(max_batch or d["kv_lens"].numel(), T, d["H"], d["page"], d["cache"].shape[0],
                   max_kv_len or max(1, int(d["kv_lens"].max())), out_dtype)


def to_cuda(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def attn(plan, d, scale=SCALE, **kw):
    return mb.mla_verify_attn_chunk(plan, d["q"], d["cache"], d["kv_indices"], d["kv_indptr"], d["kv_lens"], d["q_indptr"], scale, **kw)


def requests(d):
    """(b, first token, end token, rows, slots, which slots are in the cache) of every request."""
    ptr, first, lens = d["kv_indptr"].tolist(), d["q_indptr"].tolist(), d["kv_lens"].tolist()
    for b, n in enumerate(lens):
        slots = chunk_ref.request_slots(d["kv_indices"].numpy(), ptr, b, n, d["page"])
        yield b, first[b], first[b + 1], n, slots, (slots >= 0) & (slots < d["cache"].shape[0])


def gather(d, slots, ok):
    keys = d["cache"].double().numpy()[np.where(ok, slots, 0)]
    return np.where(ok[:, None], keys, 0.0)


# A score is the sum of 576 exact products in 36 steps of 16, each of which
# rounds (towards zero) what has been summed so far to fp32, by 2^-23 of at
# most sum |q_i k_i|.  (Twice that: the 16 products of a step are aligned and
# cut before they are added.)
SCORE_STEPS = 2 * 36


def reference(d, scale=SCALE):
    """The oracle's out and lse by token, and the bounds of their errors: a
    weight is off by its score's error and, in fp16, by 2^-11 of itself or 2^-40
    of the row's largest; lse by the score's error and the rounding of itself
    and of the logarithm (2^-22 each)."""
    N, H = d["q"].shape[:2]
    out, lse = np.zeros((N, H, 512)), np.zeros((N, H))
    out_tol, lse_tol = np.zeros((N, H, 512)), np.zeros((N, H))
    for b, t0, t1, n, slots, ok in requests(d):
        if t0 == t1:
            continue
        keys = gather(d, slots, ok)
        o, l, mass, size = chunk_ref.chunk_attn(d["q"][t0:t1].double().numpy(), keys, scale, ok)
        err = SCORE_STEPS * 2.0 ** -23 * size + 2.0 ** -22 * (np.abs(np.where(np.isfinite(l), l, 0)) + 2 * np.log2(n + 1) + 4)
        out[t0:t1], lse[t0:t1] = o, l
        lse_tol[t0:t1] = err
        # (An fp32 sum of n terms: n 2^-24 of it at the very most, in steps of 16.)
        out_tol[t0:t1] = (2.0 ** -11 + 2 * np.expm1(2 * err) + (n / 16 + 16) * 2.0 ** -23)[..., None] * mass + 2.0 ** -40 * n * 64
    return out, lse, out_tol, lse_tol


def assert_close(d, out, lse, rows=None, scale=SCALE):
    ref = reference(d, scale)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    first, end = int(d["q_indptr"][0]), int(d["q_indptr"][-1])
    rows = np.arange(first, end) if rows is None else rows
    out_tol = ref[2][rows]
    if out.dtype == torch.bfloat16:
        out_tol = out_tol + 2.0 ** -8 * np.abs(ref[0][rows])
    none = np.isneginf(l[rows]) & np.isneginf(ref[1][rows])
    eo, el = np.abs(o[rows] - ref[0][rows]), np.abs(np.where(none, 0, l[rows]) - np.where(none, 0, ref[1][rows]))
    assert (eo <= out_tol).all(), f"out: {np.max(eo / np.maximum(out_tol, 1e-30)):.3g} of the bound, {eo.max():.3g}"
    assert (el <= ref[3][rows]).all(), f"lse: {np.max(el / np.maximum(ref[3][rows], 1e-30)):.3g} of the bound, {el.max():.3g}"
