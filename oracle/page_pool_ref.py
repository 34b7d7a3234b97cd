"""Plain reference for forking and freeing requests of a counted page pool.

TEST INFRASTRUCTURE ONLY (see the package docstring): the product path never
imports this module.

The pages name neither; the reading used here: a fork shares the parent's full
pages, takes fresh ones for the rest off the end of the free list in child
order, and copies the rows of the parent's last, partial page; a free lowers
the counts and returns the pages that reach 0 in ascending order.  Failures
set flags (the library's device status bits of the same names) and never stop
the call.
"""
from __future__ import annotations

from typing import List

PAGE = 64

BAD_SLOT = 1
BAD_LEN = 2
BAD_INDPTR = 8
BAD_POOL = 64
CAPACITY = 128
BAD_REF = 1024


def fork_kv(parents, kv_indices, kv_indptr, kv_lens, caches, refs, free_pages, extra, capacity, max_kv_len):
    """(child tables, child lens, copies, refs, free pages, flags): `caches` is
    a list of lists of rows (one per layer, any objects) changed in place;
    tables are a list of lists; free_pages is the stack as a list."""
    refs, stack, flags = list(refs), list(free_pages), 0
    pages = len(refs)
    tables: List[List[int]] = []
    lens: List[int] = []
    used = 0
    stopped = False
    for p in parents:
        table, n = [], None
        if not 0 <= p < len(kv_lens):
            flags |= BAD_POOL
        elif kv_lens[p] < 0 or kv_lens[p] + extra > max_kv_len:
            flags |= BAD_LEN
        elif (kv_indptr[p] < 0 or kv_indptr[p + 1] > kv_indptr[-1]
              or (kv_indptr[p + 1] - kv_indptr[p]) * PAGE < kv_lens[p]):
            flags |= BAD_INDPTR
        else:
            n = kv_lens[p]
        if n is not None:
            total = -(-(n + extra) // PAGE)
            fresh = total - n // PAGE
            if stopped or used + total > capacity or fresh > len(stack):
                stopped = True
                if total > 0:
                    flags |= CAPACITY
                    n = None
        if n is None:
            tables.append([])
            lens.append(0)
            continue
        used += total
        for j in range(total):
            if j < n // PAGE:
                page = kv_indices[kv_indptr[p] + j]
                if 0 <= page < pages:
                    flags |= BAD_REF if refs[page] <= 0 else 0
                    refs[page] += 1
                else:
                    flags |= BAD_SLOT
            else:
                page = stack.pop()
                if 0 <= page < pages:
                    flags |= BAD_REF if refs[page] != 0 else 0
                    refs[page] = 1
                else:
                    flags |= BAD_SLOT
            table.append(page)
        if n % PAGE and 0 <= table[n // PAGE] < pages:
            src = kv_indices[kv_indptr[p] + n // PAGE]
            if not 0 <= src < pages:
                flags |= BAD_SLOT
            for rows in caches:
                for r in range(n % PAGE):
                    ok = 0 <= src < pages
                    rows[table[n // PAGE] * PAGE + r] = rows[src * PAGE + r] if ok else 0 * rows[0]
        tables.append(table)
        lens.append(n + extra)
    return tables, lens, refs, stack, flags


def free_kv(tables, refs, free_pages):
    """(refs, free pages, flags) after every table of the list ends."""
    refs, flags, gone = list(refs), 0, set()
    for table in tables:
        for page in table:
            if not 0 <= page < len(refs):
                flags |= BAD_SLOT
            elif refs[page] <= 0:
                flags |= BAD_REF
            else:
                refs[page] -= 1
                if refs[page] == 0:
                    gone.add(page)
    return refs, list(free_pages) + sorted(gone), flags
