"""Plain reference for causal attention of chunks of new tokens, in fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring): the product path never
imports this module.

The pages name no prefill; the reading used here: a request's new tokens' own
rows are the last of its cached rows, and token i of c sees the rows up to and
including its own, 0 .. n - c + i.
"""
from __future__ import annotations

import numpy as np


def request_slots(kv_indices, kv_indptr, b, n, page):
    """Slots of the n rows of request b."""
    j = np.arange(n)
    return np.asarray(kv_indices)[kv_indptr[b] + j // page].astype(np.int64) * page + j % page


def chunk_attn(q, keys, scale, visible=None):
    """Tokens q [c, H, 576] over keys [n, 576] (fp64): out [c, H, 512], lse
    [c, H], the sum of |weight * value| [c, H, 512] and the largest scale *
    sum |q_i k_i| of a row's keys [c, H] (what roundings are relative to).
    Keys that are not in `visible` (bad slots) are masked."""
    c, H, _ = q.shape
    n = keys.shape[0]
    rows = q.reshape(c * H, -1)
    s = scale * (rows @ keys.T)
    size = abs(scale) * (np.abs(rows) @ np.abs(keys).T)
    seen = np.arange(n)[None] <= (n - c + np.arange(c))[:, None]
    if visible is not None:
        seen = seen & np.asarray(visible)[None]
    seen = np.repeat(seen, H, 0)
    s = np.where(seen, s, -np.inf)
    top = s.max(1, keepdims=True)
    p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    total = p.sum(1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = (np.where(np.isfinite(top), top, 0.0) + np.log(total))[:, 0]
        p = np.where(total > 0, p / np.where(total > 0, total, 1), 0.0)
    v = keys[:, :512]
    return ((p @ v).reshape(c, H, 512), lse.reshape(c, H), (p @ np.abs(v)).reshape(c, H, 512),
            np.where(seen, size, 0).max(1).reshape(c, H))
