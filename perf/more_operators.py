"""Cases of the operators for prompts that arrive in chunks and for caches that are kept to a budget.

Three operators, in the order a serving program uses them: causal attention of any number of new tokens of each request over its
paged cache (`mla_verify_attn_chunk`), the attention weight that those tokens gave to every cached row, added up (`weigh_kv`), and
requests cut down to the rows that were given most, with the pages they leave returned to the pool (`evict_kv`).

Each case is a dict of plain values.  `run` computes it in elementary torch operations, or, where `own` is set, through this
repository's package.
"""
import math
import random

import torch

own = False

D, DV, PAGE = 576, 512, 64              # row of the cache, its value part, rows of a page
SCALE = 1.0 / math.sqrt(192.0)


def listed():
    return [
        # Attention.  Two short follow-ups to short conversations: the smallest call, where latency counts.
        dict(name="chunk_tiny", op="chunk", chunks=2, tokens=4, singles=0, cached=256, heads=16, page=1, pad=0),
        # The first chunk of a prompt: nothing is cached before it.
        dict(name="chunk_first", op="chunk", chunks=1, tokens=2048, singles=0, cached=0, heads=64, page=64, pad=0),
        # A serving step that carries a prompt's chunk beside requests that decode, padded to a captured size.
        dict(name="chunk_mixed", op="chunk", chunks=1, tokens=512, singles=23, cached=8192, heads=64, page=64, pad=9),
        # Several prompts at once, of odd lengths, with a tensor-parallel slice of the heads.
        dict(name="chunk_ragged", op="chunk", chunks=7, tokens=700, singles=0, cached=3000, heads=20, page=1, pad=0),
        # A late chunk of a long document: the largest.
        dict(name="chunk_long", op="chunk", chunks=1, tokens=2048, singles=0, cached=30720, heads=64, page=64, pad=0),
        # Weights.  Two short requests that decode: the smallest call.
        dict(name="weigh_tiny", op="weigh", chunks=0, tokens=1, singles=2, cached=256, heads=16, page=64, pad=0),
        # Every decoding step adds its token's weights: each key is read for one token's heads.
        dict(name="weigh_step", op="weigh", chunks=0, tokens=1, singles=16, cached=16384, heads=64, page=1, pad=3),
        # The last tokens of a long prompt decide what of it is kept.
        dict(name="weigh_window", op="weigh", chunks=1, tokens=32, singles=0, cached=32768, heads=64, page=64, pad=0),
        # All tokens of the chunks of several prompts.
        dict(name="weigh_prompt", op="weigh", chunks=4, tokens=256, singles=0, cached=8192, heads=32, page=1, pad=0),
        # Eviction.  One request, one layer's cache.
        dict(name="evict_one", op="evict", requests=1, rows=4096, budget=1024, sink=4, recent=64, layers=1, page=64, extra=1, fresh=0.1),
        # A batch in every layer of a cache, with room for the next drafts.
        dict(name="evict_layers", op="evict", requests=16, rows=8192, budget=2048, sink=4, recent=256, layers=16, page=64, extra=8,
             fresh=0.1),
        # A cache of single slots, where no row moves; most rows were never weighed, so that the lowest index decides.
        dict(name="evict_slots", op="evict", requests=32, rows=32768, budget=4096, sink=0, recent=100, layers=1, page=1, extra=0,
             fresh=0.9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("chunk", "chunk", "weigh", "weigh", "evict"))
    if op == "evict":
        while True:
            rows = _log(rng, 16, 32768)
            budget = _log(rng, 4, rows + 8)
            sink = rng.randint(0, budget // 4)
            case = dict(op="evict", requests=_log(rng, 1, 32), rows=rows, budget=budget, sink=sink,
                        recent=rng.randint(0, (budget - sink) // 2), layers=1, page=rng.choice((1, 64, 64)), extra=rng.choice((0, 1, 8)),
                        fresh=rng.choice((0.0, 0.1, 0.9)))
            if case["page"] == PAGE:
                case["layers"] = _log(rng, 1, 16)
            if case["requests"] * rows * case["layers"] <= 2000000:
                return case
    while True:
        chunks = rng.choice((0, 1, 1, 2, 5))
        case = dict(op=op, chunks=chunks, tokens=_log(rng, 1, 2048 if op == "chunk" else 256), singles=_log(rng, 1, 24) - 1,
                    cached=rng.choice((0, _log(rng, 1, 32768), _log(rng, 64, 16384))), heads=rng.choice((1, 8, 16, 20, 32, 64, 128)),
                    page=rng.choice((1, 64)), pad=rng.choice((0, 0, 5)))
        requests = chunks + case["singles"]
        scores = (chunks * case["tokens"] + case["singles"]) * case["heads"] * (case["cached"] + case["tokens"])
        if requests and scores <= 1e9 and requests * (case["cached"] + case["tokens"]) <= 500000:
            return case


# ---- the structure of a case: everything that is not a value, from the case alone --------------------------------------------------

def _structure(case):
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] == "evict":
        if case["requests"] == 1:
            return dict(lens=[case["rows"]])
        return dict(lens=[rng.randint(max(1, case["rows"] // 2), case["rows"]) for _ in range(case["requests"])])
    total = case["chunks"] + case["singles"]
    new = [case["tokens"] if total == 1 else rng.randint(max(1, case["tokens"] // 2), case["tokens"]) for _ in range(case["chunks"])]
    new += [1] * case["singles"]
    rng.shuffle(new)
    cached = [case["cached"] if total == 1 else rng.randint(case["cached"] // 4, case["cached"]) for _ in range(total)]
    return dict(new=new, lens=[c + n for c, n in zip(cached, new)])


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(counts):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return at


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _prepare_tokens(case, g):
    st = _structure(case)
    H, page, new, lens = case["heads"], case["page"], st["new"], st["lens"]
    entries = [-(-n // page) for n in lens]
    units = sum(entries) + max(8, sum(entries) // 8)
    if page == 1:
        units = -(-units // PAGE) * PAGE
    slots, N = units * page, sum(new) + case["pad"]
    cache = _normal(g, slots, D)
    q = _normal(g, N, H, D)
    marked = torch.rand(slots, generator=g, device="cuda")
    if case["op"] == "chunk":
        cache[marked < 0.01] *= 8                                     # a few keys stand out, as attention sinks do
    else:
        common = torch.randn(D, generator=g, device="cuda") * 0.3     # a few keys are what most queries look for
        cache[marked < 0.05] += common.to(torch.bfloat16)
        q += common.to(torch.bfloat16)
    s = dict(case=case, q=q, cache=cache, kv_indices=torch.randperm(units, generator=g, device="cuda")[:sum(entries)].to(torch.int32),
             kv_indptr=_ints(_starts(entries)), kv_lens=_ints(lens), q_indptr=_ints(_starts(new)), new=new, lens=lens)
    if case["op"] == "chunk":
        s["out"] = torch.zeros(N, H, DV, dtype=torch.bfloat16, device="cuda")     # a captured step's buffers
        s["lse"] = torch.zeros(N, H, dtype=torch.float32, device="cuda")
    else:
        s["lse"] = _plain_attn(s, None, torch.zeros(N, H, device="cuda"))         # as the step's attention left it
        s["weights"] = torch.rand(len(lens), max(lens) + 100, generator=g, device="cuda")
        s["weights"] *= torch.arange(s["weights"].shape[1], device="cuda") < (s["kv_lens"] - _ints(new))[:, None]   # new rows: 0
    if own:
        from paged_mla_speculative_gb300 import binding
        s["binding"] = binding
        s["plan"] = binding.Plan(len(lens), 1, H, page, slots, max(lens), torch.bfloat16)
    return s


def _prepare_evict(case, g):
    lens = _structure(case)["lens"]
    B, page, budget, extra = len(lens), case["page"], case["budget"], case["extra"]
    counts = [-(-n // page) for n in lens]
    after = [-(-(min(n, budget) + extra) // page) for n in lens]
    units = -(-(sum(counts) + sum(after) + 8) // PAGE) * PAGE
    ids = torch.randperm(units, generator=g, device="cuda").to(torch.int32)
    pool = torch.zeros(2 * units + 4, dtype=torch.int32, device="cuda")           # counts, stack of free pages, its height
    pool[:units][ids[:sum(counts)].long()] = 1
    pool[units:units + units - sum(counts)] = ids[sum(counts):]
    pool[2 * units] = units - sum(counts)
    held = pool[:units]
    held[ids[:sum(counts) // 16].long()] += 1                                     # some pages are in other requests' tables too
    width = max(lens) + 100
    weights = torch.empty(B, width, device="cuda").exponential_(generator=g)
    weights *= torch.rand(B, width, generator=g, device="cuda") >= case["fresh"]  # rows that no token has weighed yet: 0
    s = dict(case=case, lens=lens, weights=weights, pool=pool, pool_before=pool.clone(), refs=held, free=pool[units:2 * units],
             count=pool[2 * units:2 * units + 1], indices=ids[:sum(counts)].clone(), indptr=_ints(_starts(counts)), kv_lens=_ints(lens),
             cache=torch.randn(case["layers"], units * page, D, generator=g, device="cuda", dtype=torch.bfloat16) if page > 1 else None,
             new_indices=torch.full((sum(after) + 5,), -7, dtype=torch.int32, device="cuda"), new_indptr=_ints([0] * (B + 1)),
             new_lens=_ints([0] * B), new_weights=torch.full((B, width), -7.0, device="cuda"), after=max(after))
    if own:
        from paged_mla_speculative_gb300 import binding
        s["binding"] = binding
        s["plan"] = binding.Plan(B, 1, 16, page, units * page, max(lens) + extra, torch.bfloat16)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return _prepare_evict(case, g) if case["op"] == "evict" else _prepare_tokens(case, g)


# ---- plain forms ---------------------------------------------------------------------------------------------------------------------

def _scores(s):
    """For each number of new tokens that requests have: those requests [R], their tokens [R, c], the scores [R, c, H, L] (-inf where
    a token does not see a key) and the keys [R, L, D]."""
    page, H = s["case"]["page"], s["case"]["heads"]
    for c in sorted(set(s["new"])):
        same = [b for b, n in enumerate(s["new"]) if n == c]
        r = torch.tensor(same, device="cuda")
        L = max(s["lens"][b] for b in same)
        n = s["kv_lens"].long()[r][:, None]
        j = torch.arange(L, device="cuda")[None]
        jj = torch.minimum(j, n - 1)
        k = s["cache"][s["kv_indices"][s["kv_indptr"].long()[r][:, None] + jj // page].long() * page + jj % page].float()
        i = torch.arange(c, device="cuda")
        at = s["q_indptr"].long()[r][:, None] + i
        x = torch.matmul(s["q"][at].float().reshape(len(same), c * H, D), k.transpose(1, 2)).reshape(len(same), c, H, L)
        x *= SCALE
        x.masked_fill_((j[:, None] > (n - c + i)[..., None])[:, :, None], -math.inf)
        yield r, at, x, k


def _plain_attn(s, out, lse):
    for r, at, x, k in _scores(s):
        m = x.amax(-1, keepdim=True)
        x -= m
        x.exp_()
        l = x.sum(-1, keepdim=True)
        lse[at] = (m + torch.log(l))[..., 0]
        if out is not None:
            R, c, H, L = x.shape
            out[at] = (torch.matmul(x.reshape(R, c * H, L), k[..., :DV]).reshape(R, c, H, DV) / l).to(out.dtype)
    return lse


def _plain_weigh(s):
    for r, at, x, k in _scores(s):
        x -= s["lse"][at][..., None]
        x.exp_()
        s["weights"][r, :x.shape[-1]] += x.sum((1, 2))


def _plain_evict(s):
    case, page = s["case"], s["case"]["page"]
    budget, extra = case["budget"], case["extra"]
    B, width = s["weights"].shape
    n = s["kv_lens"].long()[:, None]
    m = n.clamp(max=budget)
    j = torch.arange(width, device="cuda")[None]
    w = s["weights"].masked_fill((j < case["sink"]) | (j >= n - case["recent"]) | (n <= budget), math.inf).masked_fill(j >= n, -math.inf)
    rank = torch.empty_like(w, dtype=torch.int64)
    rank.scatter_(1, w.sort(dim=1, descending=True, stable=True).indices, j.expand(B, width))    # equal weights: the lowest index first
    kept = (rank < m) & (j < n)
    first = torch.argsort((~kept).to(torch.uint8), dim=1, stable=True)               # the kept rows in their order, then the others
    s["new_weights"].copy_(s["weights"].gather(1, first).masked_fill(j >= m, 0.0))
    # Entries: those that stay (single slots: the kept ones; pages: all of a request that is within the budget, else the leading ones
    # that hold protected rows alone), then fresh ones off the end of the free list.
    whole = n <= budget
    stay = m if page == 1 else torch.where(whole, (n + page - 1) // page, case["sink"] // page)
    total = torch.maximum((m + extra + page - 1) // page, stay)
    ends = total[:, 0].cumsum(0)
    fresh = (total - stay)[:, 0]
    before = (fresh.cumsum(0) - fresh)[:, None]
    left = s["count"].long()
    e = torch.arange(max(s["after"], 1), device="cuda")[None]
    start = s["indptr"].long()[:-1][:, None]
    old = first.gather(1, e.clamp(max=width - 1).expand(B, -1)) if page == 1 else e
    mine = s["indices"][(start + torch.minimum(old, (n + page - 1) // page - 1)).clamp(0)].long()
    taken = s["free"][(left - 1 - (before + (e - stay).clamp(0))).clamp(0)].long()
    entry = torch.where(e < stay, mine, taken)
    used = e < total
    room = torch.cat((s["new_indices"], s["new_indices"][:1]))                       # one more place, for what is not written
    room[torch.where(used, ends[:, None] - total + e, s["new_indices"].numel())] = entry.to(torch.int32)
    s["new_indices"].copy_(room[:-1])
    s["new_indptr"].copy_(torch.cat((ends.new_zeros(1), ends)))
    s["new_lens"].copy_((m + extra)[:, 0])
    if page > 1:                                                                     # kept rows behind the entries that stay
        i = torch.arange(budget, device="cuda")[None]
        moves = (i >= stay * page) & (i < m) & ~whole
        source = first[:, :budget] if width >= budget else torch.cat((first, first[:, :1].expand(B, budget - width)), 1)
        src = s["indices"][start + torch.minimum(source, n - 1) // page].long() * page + source % page
        dst = entry.gather(1, (i // page).clamp(max=e.shape[1] - 1).expand(B, -1)) * page + i % page
        src, dst = src[moves], dst[moves]
        s["cache"][:, dst] = s["cache"][:, src]
    # Counts: fresh entries 1, entries that were left one less; those that fall to 0 go back in ascending order.
    s["refs"].index_add_(0, entry.flatten(), (used & (e >= stay)).flatten().to(torch.int32))
    had = s["refs"].clone()
    t = torch.arange(s["indices"].numel(), device="cuda")
    b = torch.searchsorted(s["indptr"].long()[1:], t, right=True)
    place = t - s["indptr"].long()[b]
    gone = ~kept[b, place.clamp(max=width - 1)] if page == 1 else (place >= stay[b, 0]) & ~whole[b, 0]
    s["refs"].index_add_(0, s["indices"].long(), -gone.to(torch.int32))
    empty = (had > 0) & (s["refs"] == 0)
    left = left - fresh.sum()
    at = torch.where(empty, left + empty.cumsum(0) - 1, s["free"].numel())
    room = torch.cat((s["free"], s["free"][:1]))
    room[at] = torch.arange(s["free"].numel(), device="cuda", dtype=torch.int32)
    s["free"].copy_(room[:-1])
    s["count"].copy_(left + empty.sum())


# ---- one pass ------------------------------------------------------------------------------------------------------------------------

def run(state):
    s = state
    op = s["case"]["op"]
    if op == "chunk":
        if own:
            s["binding"].mla_verify_attn_chunk(s["plan"], s["q"], s["cache"], s["kv_indices"], s["kv_indptr"], s["kv_lens"],
                                               s["q_indptr"], SCALE, out=s["out"], lse=s["lse"])
        else:
            _plain_attn(s, s["out"], s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "weigh":
        if own:
            s["binding"].weigh_kv(s["plan"], s["q"], s["cache"], s["kv_indices"], s["kv_indptr"], s["kv_lens"], s["q_indptr"],
                                  s["lse"], SCALE, s["weights"])
        else:
            _plain_weigh(s)
        return {"weights": s["weights"]}
    s["pool"].copy_(s["pool_before"])                                # a pass begins with the pool that its tables belong to
    if own:
        s["binding"].evict_kv(s["plan"], s["weights"], s["case"]["budget"], s["indices"], s["indptr"], s["kv_lens"], s["cache"],
                              s["refs"], s["free"], s["count"], sink=s["case"]["sink"], recent=s["case"]["recent"],
                              extra_rows=s["case"]["extra"], new_indices=s["new_indices"], new_indptr=s["new_indptr"],
                              new_lens=s["new_lens"], new_weights=s["new_weights"])
    else:
        _plain_evict(s)
    got = {"indices": s["new_indices"], "indptr": s["new_indptr"], "lens": s["new_lens"], "weights": s["new_weights"], "refs": s["refs"],
           "free": s["free"], "count": s["count"]}
    if s["cache"] is not None:
        got["cache"] = s["cache"]
    return got


def work(case):
    st = _structure(case)
    if case["op"] == "evict":
        entries = moved = weights = 0
        for n in st["lens"]:
            m = min(n, case["budget"])
            entries += -(-n // case["page"]) + -(-(m + case["extra"]) // case["page"])
            weights += n + m
            if case["page"] > 1 and n > m:
                moved += m - case["sink"] // PAGE * PAGE
        # a weight read, and one written for each row that is kept; an entry with its count read and written; rows both ways
        return {"bytes": 4 * weights + 12 * entries + moved * case["layers"] * D * 2 * 2, "flops": 0}
    H = case["heads"]
    keys, tokens = sum(st["lens"]), sum(st["new"])
    pairs = sum(c * (n - c) + c * (c + 1) // 2 for c, n in zip(st["new"], st["lens"])) * H
    if case["op"] == "chunk":
        return {"bytes": tokens * H * (D * 2 + DV * 2 + 4) + keys * D * 2, "flops": 2.0 * (D + DV) * pairs}
    return {"bytes": tokens * H * (D * 2 + 4) + keys * (D * 2 + 8), "flops": 2.0 * D * pairs}


# ---- the definition, in 64 bits ------------------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "evict":
        return None                                                  # rows are chosen, moved and counted: no computed numbers
    if work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    H, page = case["heads"], case["page"]
    if case["op"] == "chunk":
        out, lse = s["out"].double(), s["lse"].double()
    else:
        weights = s["weights"].double()
    table, starts, firsts = s["kv_indices"].long(), s["kv_indptr"].tolist(), s["q_indptr"].tolist()
    for b, (n, c) in enumerate(zip(s["lens"], s["new"])):
        slots = (table[starts[b]:starts[b + 1], None] * page + torch.arange(page, device="cuda")).flatten()[:n]
        keys = s["cache"][slots].double()
        step = max(1, 200000000 // (n * H))
        for t0 in range(0, c, step):
            t1 = min(c, t0 + step)
            rows = slice(firsts[b] + t0, firsts[b] + t1)
            sees = torch.tril(torch.ones(t1 - t0, n, dtype=torch.bool, device="cuda"), n - c + t0)[:, None]
            z = torch.einsum("thd,nd->thn", s["q"][rows].double(), keys) * SCALE
            if case["op"] == "chunk":
                z = torch.where(sees, z, -math.inf)
                lse[rows] = torch.logsumexp(z, -1)
                out[rows] = torch.einsum("thn,nd->thd", torch.softmax(z, -1), keys[:, :DV])
            else:
                weights[b, :n] += torch.where(sees, torch.exp(z - s["lse"][rows].double()[..., None]), 0.0).sum((0, 1))
    return {"out": out, "lse": lse} if case["op"] == "chunk" else {"weights": weights}
