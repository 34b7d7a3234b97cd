"""Plain reference for weighing and evicting cached rows.

TEST INFRASTRUCTURE ONLY (see the package docstring): the product path never
imports this module.

The pages name neither; the reading used here: a row's weight is the sum, over
all new tokens and heads that see it, of the softmax weight that they give it;
a request that holds more rows than the budget keeps its first `sink` rows, its
last `recent` rows and of the others those with the largest weights, the lowest
index first among equals (-0 equals 0, NaN is below every number), all in their
order.  Failures set flags (the library's device status bits of the same names)
and never stop the call.
"""
from __future__ import annotations

import math

import numpy as np

BAD_SLOT = 1
BAD_LEN = 2
BAD_INDPTR = 8
CAPACITY = 128
BAD_REF = 1024


def weigh(q, keys, lse, scale, visible=None):
    """What rows q [c, H, 576] with log-sum-exps lse [c, H] give each of keys
    [n, 576] (fp64): token i sees keys 0 .. n - c + i.  A row whose lse is not
    finite gives nothing; a key that is not in `visible` gets nothing."""
    c, n = q.shape[0], keys.shape[0]
    w = np.zeros(n)
    for i in range(c):
        for h in range(q.shape[1]):
            if not math.isfinite(lse[i, h]):
                continue
            for j in range(n - c + i + 1):
                if visible is None or visible[j]:
                    w[j] += math.exp(scale * float(np.dot(q[i, h], keys[j])) - lse[i, h])
    return w


def keep(weights, n, budget, sink, recent):
    """The kept rows of a request of n rows, ascending."""
    if n <= budget:
        return list(range(n))
    held = set(range(sink)) | set(range(n - recent, n))
    rest = [j for j in range(n) if j not in held]

    def order(j):
        w = float(weights[j])
        return (1, 0.0, j) if math.isnan(w) else (0, -w, j)

    return sorted(held | set(sorted(rest, key=order)[:budget - len(held)]))


def evict_kv(weights, budget, sink, recent, extra, page, kv_indices, kv_indptr, kv_lens, caches, refs, free_pages, capacity,
             max_kv_len):
    """(tables, lens, weights, refs, free pages, flags): `weights` is a list of
    rows; `caches` a list of lists of rows (one per layer, any objects) changed
    in place, not used with page 1; tables a list of lists; free_pages the
    stack as a list."""
    refs, stack, flags, gone = list(refs), list(free_pages), 0, set()
    units = len(refs)
    tables, lens, out = [], [], []
    used = 0
    stopped = False
    for b, n in enumerate(kv_lens):
        p0, p1 = kv_indptr[b], kv_indptr[b + 1]
        table, new_len, row = [], 0, [0.0] * len(weights[b])
        ok = False
        if n < 0 or n > max_kv_len or min(n, budget) + extra > max_kv_len:
            flags |= BAD_LEN
        elif p0 < 0 or p1 > kv_indptr[-1] or (p1 - p0) * page < n:
            flags |= BAD_INDPTR
        else:
            ok = True
        if ok:
            kept = keep(weights[b], n, budget, sink, recent)
            old = list(kv_indices[p0:p1])
            if page == 1:
                stay = [old[j] for j in kept]
                stays = set(kept)
                left = [old[j] for j in range(len(old)) if j not in stays]
            else:
                count = -(-n // page) if n <= budget else sink // page
                stay, left = old[:count], old[count:]
            total = max(-(-(len(kept) + extra) // page), len(stay))
            if stopped or used + total > capacity or total - len(stay) > len(stack):
                stopped = True
                if total > 0 or left:
                    flags |= CAPACITY
                ok = False
        if ok:
            used += total
            fresh = [stack.pop() for _ in range(total - len(stay))]
            for u in fresh:
                if 0 <= u < units:
                    flags |= BAD_REF if refs[u] != 0 else 0
                    refs[u] = 1
                else:
                    flags |= BAD_SLOT
            table = stay + fresh
            for u in stay:
                if not 0 <= u < units:
                    flags |= BAD_SLOT
            if page > 1 and n > budget:
                for i in range(len(stay) * page, len(kept)):
                    src, dst = old[kept[i] // page], table[i // page]
                    if not 0 <= src < units:
                        flags |= BAD_SLOT
                    if 0 <= dst < units:
                        for rows in caches:
                            ok_src = 0 <= src < units
                            rows[dst * page + i % page] = rows[src * page + kept[i] % page] if ok_src else 0 * rows[0]
            for u in left:
                if not 0 <= u < units:
                    flags |= BAD_SLOT
                elif refs[u] <= 0:
                    flags |= BAD_REF
                else:
                    refs[u] -= 1
                    if refs[u] == 0:
                        gone.add(u)
            new_len = len(kept) + extra
            row = [weights[b][j] for j in kept] + [0.0] * (len(weights[b]) - len(kept))
        tables.append(table)
        lens.append(new_len)
        out.append(row)
    return tables, lens, out, refs, stack + sorted(gone), flags
