"""Plain reference for new tokens' cache rows and queries, in fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring): the product path never
imports this module.

The pages name no procedure for writing rows; the reading used here is MLA's:
the latent is divided by its root mean square and scaled, the 64 shared rope
dims and every query head's are rotated by the token's position, pair by pair:
neighbours (2i, 2i + 1), or halves (i, i + 32).
"""
from __future__ import annotations

import numpy as np

BAD_SLOT = 1
BAD_POS = 512


def rotate(x: np.ndarray, cos_sin: np.ndarray, halves: bool) -> np.ndarray:
    """x [64] turned by the 32 angles whose cosines and sines are cos_sin [64]."""
    y = np.empty(64)
    for i in range(32):
        a, b = (i, i + 32) if halves else (2 * i, 2 * i + 1)
        c, s = cos_sin[i], cos_sin[32 + i]
        y[a] = x[a] * c - x[b] * s
        y[b] = x[b] * c + x[a] * s
    return y


def append_kv(kv, weight, eps, q_nope, q_pe, cos_sin, positions, slots, halves, cache, q):
    """(cache, q, flags) after the call, in fp64; inputs are fp64 arrays (cache
    and q as they were before), q_nope None where q holds it already."""
    cache, q, flags = np.array(cache), np.array(q), 0
    for n in range(len(slots)):
        s, p = int(slots[n]), int(positions[n])
        if s == -1:
            continue
        slot_ok, pos_ok = 0 <= s < cache.shape[0], 0 <= p < cos_sin.shape[0]
        if not (slot_ok and pos_ok):
            flags |= (0 if slot_ok else BAD_SLOT) | (0 if pos_ok else BAD_POS)
            continue
        c = kv[n, :512]
        cache[s, :512] = c / np.sqrt(np.dot(c, c) / 512 + eps) * weight
        cache[s, 512:] = rotate(kv[n, 512:], cos_sin[p], halves)
        for h in range(q.shape[1]):
            if q_nope is not None:
                q[n, h, :512] = q_nope[n, h]
            q[n, h, 512:] = rotate(q_pe[n, h], cos_sin[p], halves)
    return cache, q, flags
