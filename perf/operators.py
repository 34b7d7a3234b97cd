"""Cases of the operators for a cached prompt that many requests share.

Four operators, in the order a serving program uses them: new tokens' keys normalised, rotated and written into the paged latent
cache with their queries assembled (`append_kv`), requests branching off a cached one by sharing its full pages (`fork_kv`) and
ending again (`free_kv`), and the verify attention of a batch whose groups of requests share their first rows
(`mla_verify_attn_shared`).

Each case is a dict of plain values.  `run` computes it in elementary torch operations, or, where `own` is set, through this
repository's package.
"""
import math
import random

import torch

own = False

D, DV, DR, PAGE = 576, 512, 64, 64      # row of the cache, its value part, its rotated part, rows of a page
SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6


def listed():
    return [
        # Attention.  Two requests on a short system prompt: the smallest call, where latency counts.
        dict(name="shared_tiny", op="attn", groups=1, requests=2, drafts=4, heads=16, shared=256, own_rows=24, page=1, tree=False),
        # One new token each for 64 samples of one prompt: decoding without drafts.
        dict(name="shared_decode", op="attn", groups=1, requests=64, drafts=1, heads=128, shared=2048, own_rows=512, page=64, tree=False),
        # The ordinary verify step of eight requests on one long context, eight chained drafts each.
        dict(name="shared_verify", op="attn", groups=1, requests=8, drafts=8, heads=64, shared=16384, own_rows=200, page=1, tree=False),
        # Four prompts with branches of their own, a tensor-parallel slice of the heads, draft trees: few rows for each key.
        dict(name="shared_groups", op="attn", groups=4, requests=23, drafts=4, heads=16, shared=8192, own_rows=1000, page=64, tree=True),
        # Sixteen requests on a book-length context with trees of sixteen drafts: the largest.
        dict(name="shared_long", op="attn", groups=1, requests=16, drafts=16, heads=64, shared=65536, own_rows=500, page=64, tree=True),
        # New rows.  One verify step's drafts: eight requests, eight drafts.
        dict(name="append_step", op="append", tokens=64, heads=64, pad=0, interleaved=True, absorbed=True, max_pos=16384),
        # A prompt's chunk: keys and the queries of every head.
        dict(name="append_prompt", op="append", tokens=8192, heads=64, pad=0, interleaved=True, absorbed=True, max_pos=65536),
        # A padded, captured batch of odd size whose absorbed queries are already in place; the two halves rotated.
        dict(name="append_padded", op="append", tokens=1003, heads=16, pad=101, interleaved=False, absorbed=False, max_pos=16384),
        # Pages.  Four samples started on one prompt and dropped again, one layer's cache.
        dict(name="fork_samples", op="fork", parents=1, children=4, rows=300, extra=4, layers=1, beam=False),
        # Sixty-four branches of eight prompts, in every layer of a cache.
        dict(name="fork_layers", op="fork", parents=8, children=64, rows=4000, extra=8, layers=16, beam=False),
        # A beam step: the survivors' branches take the places of all beams.
        dict(name="beam_step", op="fork", parents=16, children=16, rows=1000, extra=0, layers=4, beam=True),
        # The same on long contexts: the tables are what is large.
        dict(name="beam_long", op="fork", parents=32, children=32, rows=30000, extra=0, layers=1, beam=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("attn", "attn", "append", "fork"))
    if kind == "attn":
        while True:
            groups = rng.choice((1, 1, 2, 3, 4))
            case = dict(op="attn", groups=groups, requests=groups + _log(rng, 1, 48) - 1, drafts=_log(rng, 1, 16),
                        heads=rng.choice((8, 16, 20, 32, 64, 128)), shared=_log(rng, 64, 32768), own_rows=_log(rng, 24, 1000),
                        page=rng.choice((1, 64)), tree=rng.random() < 0.5)
            rows = case["requests"] * case["drafts"] * case["heads"]
            if case["drafts"] * case["heads"] <= 4096 and rows * (case["shared"] + case["own_rows"]) <= 4e8:
                return case
    if kind == "append":
        tokens = _log(rng, 1, 8192)
        heads = rng.choice((8, 16, 20, 32, 64))
        return dict(op="append", tokens=tokens, heads=heads, pad=rng.choice((0, tokens // 7)), interleaved=rng.random() < 0.5,
                    absorbed=rng.random() < 0.7, max_pos=_log(rng, 8192, 65536))
    beam = rng.random() < 0.5
    parents = _log(rng, 1, 32)
    rows = _log(rng, 1, 16000)
    layers = _log(rng, 1, 16)
    while parents * rows * layers > 500000:
        layers, rows = max(1, layers // 2), rows if layers > 1 else rows // 2
    return dict(op="fork", parents=parents, children=parents if beam else _log(rng, 1, 64), rows=rows,
                extra=0 if beam else rng.choice((0, 1, 8)), layers=layers, beam=beam)


# ---- the structure of a case: everything that is not a value, from the case alone --------------------------------------------------

def _structure(case):
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] == "attn":
        G, B, T = case["groups"], case["requests"], case["drafts"]
        cuts = sorted(rng.sample(range(1, B), G - 1)) if G > 1 else []
        group_indptr = [0] + cuts + [B]
        shared = [case["shared"] if G == 1 else rng.randint(max(1, case["shared"] // 4), case["shared"]) for _ in range(G)]
        if case["page"] == PAGE:   # branches share whole pages
            shared = [max(PAGE, s // PAGE * PAGE) for s in shared]
        lens = [rng.randint(T, max(T, case["own_rows"])) for _ in range(B)]
        group = [g for g in range(G) for _ in range(group_indptr[g], group_indptr[g + 1])]
        return dict(group_indptr=group_indptr, shared=shared, own=lens, group=group,
                    kv_lens=[shared[group[b]] + lens[b] for b in range(B)])
    if case["op"] == "fork":
        n = [rng.randint(max(1, case["rows"] // 2), case["rows"]) for _ in range(case["parents"])]
        parents = sorted(rng.randrange(case["parents"]) for _ in range(case["children"]))
        return dict(lens=n, parents=parents)
    return {}


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _prepare_attn(case, g):
    st = _structure(case)
    B, T, H, page = case["requests"], case["drafts"], case["heads"], case["page"]
    up = (lambda n: n) if page == 1 else (lambda n: -(-n // PAGE))
    entries = [up(n) for n in st["kv_lens"]]
    shared_entries = [s if page == 1 else s // PAGE for s in st["shared"]]
    need = sum(shared_entries) + sum(e - shared_entries[st["group"][b]] for b, e in enumerate(entries))
    units = need + max(8, need // 8)
    if page == 1:
        units = -(-units // PAGE) * PAGE
    ids = torch.randperm(units, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    heads, at = [], 0
    for e in shared_entries:
        heads.append(ids[at:at + e])
        at += e
    table = []
    for b, e in enumerate(entries):
        k = e - shared_entries[st["group"][b]]
        table += [heads[st["group"][b]], ids[at:at + k]]
        at += k
    slots = units * page
    cache = _normal(g, slots, D)
    spiky = torch.rand(slots, generator=g, device="cuda") < 0.01      # a few keys stand out, as attention sinks do
    cache[spiky] *= 8
    if case["tree"]:
        parent = torch.floor(torch.rand(B, T, generator=g, device="cuda") * (torch.arange(T, device="cuda") + 1)).to(torch.int32) - 1
    else:
        parent = (torch.arange(T, dtype=torch.int32, device="cuda") - 1).repeat(B, 1)
    indptr = [0]
    for e in entries:
        indptr.append(indptr[-1] + e)
    s = dict(case=case, q=_normal(g, B, T, H, D), cache=cache, kv_indices=torch.cat(table), kv_indptr=_ints(indptr),
             kv_lens=_ints(st["kv_lens"]), parent=parent.contiguous(), group_indptr=_ints(st["group_indptr"]),
             shared_lens=_ints(st["shared"]), longest=max(st["kv_lens"]))
    if own:
        from paged_mla_speculative_gb300 import binding
        s["binding"] = binding
        s["plan"] = binding.Plan(B, T, H, page, slots, s["longest"], torch.bfloat16)
    return s


def _prepare_append(case, g):
    N, H = case["tokens"], case["heads"]
    slots = -(-(N + N // 4 + 8) // PAGE) * PAGE
    place = torch.randperm(slots, generator=g, device="cuda", dtype=torch.int64)[:N].to(torch.int32)
    real = N - case["pad"]
    place[real:] = -1                                               # the batch's padding comes last
    t = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)
    angle = t[:, None] * 10000.0 ** (-torch.arange(0, DR, 2, device="cuda", dtype=torch.float64) / DR)
    cos_sin = torch.cat((angle.cos(), angle.sin()), -1).float()
    pos = torch.randint(0, case["max_pos"], (N,), generator=g, device="cuda").to(torch.int32)
    fused = _normal(g, N, 1536 + D) * 3                             # the down projection's output: queries' latent, then the key's
    wide = _normal(g, N, H, 128 + DR)                               # the query up projection's output: its last dims are rotated
    s = dict(case=case, kv=fused[:, 1536:], q_pe=wide[..., 128:], q_nope=_normal(g, N, H, DV) if case["absorbed"] else None,
             weight=(1 + 0.2 * torch.randn(DV, generator=g, device="cuda")).to(torch.bfloat16), cos_sin=cos_sin, pos=pos,
             slots=place, cache=_normal(g, slots, D), q=_normal(g, N, H, D))
    if own:
        from paged_mla_speculative_gb300 import binding
        s["binding"] = binding
        s["plan"] = binding.Plan(1, 1, H, PAGE, slots, PAGE, torch.bfloat16)
    return s


def _prepare_fork(case, g):
    st = _structure(case)
    counts = [-(-n // PAGE) for n in st["lens"]]
    fresh = sum(-(-(st["lens"][p] + case["extra"]) // PAGE) - st["lens"][p] // PAGE for p in st["parents"])
    pages = sum(counts) + 2 * fresh + 2 * case["children"] + 8
    ids = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    live = sum(counts)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[ids[:live].long()] = 1
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:pages - live] = ids[live:]
    indptr = [0]
    for c in counts:
        indptr.append(indptr[-1] + c)
    most = max(-(-(n + case["extra"]) // PAGE) for n in st["lens"])
    room = max(most * case["children"], live)
    cache = torch.randn(case["layers"], pages * PAGE, D, generator=g, device="cuda", dtype=torch.bfloat16)
    indices = torch.full((room,), -7, dtype=torch.int32, device="cuda")
    indices[:live] = ids[:live]
    s = dict(case=case, cache=cache, refs=refs, free=free, count=_ints([pages - live]), parents=_ints(st["parents"]),
             table=(indices, _ints(indptr), _ints(st["lens"])),
             other=(torch.full((room,), -7, dtype=torch.int32, device="cuda"), _ints([0] * (case["children"] + 1)),
                    _ints([0] * case["children"])),
             pages=pages, most=most)
    if own:
        from paged_mla_speculative_gb300 import binding
        s["binding"] = binding
        s["plan"] = binding.Plan(max(case["parents"], case["children"]), 1, 16, PAGE, pages * PAGE,
                                 max(st["lens"]) + case["extra"] + 1, torch.bfloat16)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"attn": _prepare_attn, "append": _prepare_append, "fork": _prepare_fork}[case["op"]](case, g)


# ---- plain forms ---------------------------------------------------------------------------------------------------------------------

def _plain_attn(s):
    B, T, H, _ = s["q"].shape
    page, L = s["case"]["page"], s["longest"]
    n = s["kv_lens"].long()[:, None]
    j = torch.arange(L, device="cuda")[None]
    jj = torch.minimum(j, n - 1)
    entry = s["kv_indices"][s["kv_indptr"][:-1].long()[:, None] + jj // page].long()
    k = s["cache"][entry * page + jj % page].float()                 # [B, L, D]
    parent = s["parent"].long()
    up = torch.zeros(B, T, T + 1, device="cuda").scatter_(2, (parent % (T + 1))[..., None], 1.0)[..., :T]
    seen = torch.linalg.matrix_power(up + torch.eye(T, device="cuda"), T) > 0.5          # draft t sees draft i
    draft = j - (n - T)                                              # [B, L]
    ok = seen.gather(2, draft.clamp(0, T - 1)[:, None].expand(B, T, L)) | (draft < 0)[:, None]
    ok &= (j < n)[:, None]
    x = torch.matmul(s["q"].float().reshape(B, T * H, D), k.transpose(1, 2)).reshape(B, T, H, L) * SCALE
    x.masked_fill_(~ok[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x - m)
    l = x.sum(-1, keepdim=True)
    out = torch.matmul(x.reshape(B, T * H, L), k[..., :DV]).reshape(B, T, H, DV) / l
    return out.to(torch.bfloat16), (m + torch.log(l))[..., 0]


def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    a, b = x[..., :DR // 2], x[..., DR // 2:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _plain_append(s):
    N = s["pos"].numel()
    cs = s["cos_sin"][s["pos"].long()]
    cos, sin = cs[:, :DR // 2], cs[:, DR // 2:]
    kv = s["kv"].float()
    c = kv[:, :DV]
    c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    row = torch.cat((c, _rotate(kv[:, DV:], cos, sin, s["case"]["interleaved"])), -1).to(torch.bfloat16)
    real = s["slots"] >= 0
    first = real.int().argmax()                                      # padding repeats the first real token's write
    at = torch.where(real, torch.arange(N, device="cuda"), first)
    s["cache"][s["slots"][at].long()] = row[at]
    pe = _rotate(s["q_pe"].float(), cos[:, None], sin[:, None], s["case"]["interleaved"]).to(torch.bfloat16)
    nope = s["q"][..., :DV] if s["q_nope"] is None else s["q_nope"]
    s["q"].copy_(torch.where(real[:, None, None], torch.cat((nope, pe), -1), s["q"]))
    return s["q"], s["cache"]


def _plain_fork(s, table, to):
    """Children of `table` into `to`: full pages shared, the partial page's rows copied, fresh pages off the end of the free list."""
    indices, indptr, lens = table
    p, extra = s["parents"].long(), s["case"]["extra"]
    n = lens[p].long()
    full, total = n // PAGE, (n + extra + PAGE - 1) // PAGE
    ends = total.cumsum(0)
    new = total - full
    before = new.cumsum(0) - new
    j = torch.arange(s["most"], device="cuda")[None]
    mine, kept = j < total[:, None], j < full[:, None]
    held = indices[(indptr[p].long()[:, None] + torch.minimum(j, ((n + PAGE - 1) // PAGE)[:, None] - 1))].long()
    left = s["count"].long()
    taken = s["free"][(left - 1 - (before[:, None] + (j - full[:, None]).clamp(0))).clamp(0)].long()
    page = torch.where(kept, held, taken)
    room = torch.cat((to[0], to[0][:1]))                             # one more place, for what is not written
    room[torch.where(mine, ends[:, None] - total[:, None] + j, to[0].numel())] = page.to(torch.int32)
    to[0].copy_(room[:-1])
    to[1].copy_(torch.cat((ends.new_zeros(1), ends)))
    to[2].copy_(n + extra)
    s["refs"].index_add_(0, page.flatten(), mine.flatten().to(torch.int32))
    s["count"].sub_(new.sum().to(torch.int32))
    r = torch.arange(PAGE, device="cuda")[None]
    last = full.clamp(max=s["most"] - 1)[:, None]
    src = (held.gather(1, last) * PAGE + r)
    dst = torch.where(r < (n % PAGE)[:, None], page.gather(1, last) * PAGE + r, src)     # a row that stays is put where it is
    s["cache"][:, dst.flatten()] = s["cache"][:, src.flatten()]


def _plain_free(s, table):
    indices, indptr, _ = table
    had = s["refs"].clone()
    j = torch.arange(indices.numel(), device="cuda")
    mine = (j < indptr[-1]).to(torch.int32)
    s["refs"].index_add_(0, torch.where(mine > 0, indices, 0).long(), -mine)
    gone = (had > 0) & (s["refs"] == 0)
    at = s["count"].long() + gone.cumsum(0) - 1
    room = torch.cat((s["free"], s["free"][:1]))
    room[torch.where(gone, at, s["pages"])] = torch.arange(s["pages"], device="cuda", dtype=torch.int32)
    s["free"].copy_(room[:-1])
    s["count"].add_(gone.sum().to(torch.int32))


# ---- one pass ------------------------------------------------------------------------------------------------------------------------

def run(state):
    s = state
    op = s["case"]["op"]
    if op == "attn":
        if own:
            out, lse = s["binding"].mla_verify_attn_shared(
                s["plan"], s["q"], s["cache"], s["kv_indices"], s["kv_indptr"], s["kv_lens"], s["parent"], SCALE,
                s["group_indptr"], s["shared_lens"])
        else:
            out, lse = _plain_attn(s)
        return {"out": out, "lse": lse}
    if op == "append":
        if own:
            s["binding"].append_kv(s["plan"], s["kv"], s["weight"], EPS, s["cos_sin"], s["pos"], s["slots"], s["cache"],
                                   q_nope=s["q_nope"], q_pe=s["q_pe"], q=s["q"], interleaved=s["case"]["interleaved"])
            return {"q": s["q"], "cache": s["cache"]}
        q, cache = _plain_append(s)
        return {"q": q, "cache": cache}
    table, to = s["table"], s["other"]
    gone = table if s["case"]["beam"] else to                        # a beam step drops the old beams, a sample ends itself
    if own:
        s["binding"].fork_kv(s["plan"], s["parents"], *table, s["cache"], s["refs"], s["free"], s["count"],
                             extra_rows=s["case"]["extra"], child_indices=to[0], child_indptr=to[1], child_lens=to[2])
        s["binding"].free_kv(s["plan"], gone[0], gone[1], s["refs"], s["free"], s["count"])
    else:
        _plain_fork(s, table, to)
        _plain_free(s, gone)
    if s["case"]["beam"]:
        s["table"], s["other"] = to, table
    return {"indices": to[0], "indptr": to[1], "lens": to[2], "cache": s["cache"], "refs": s["refs"], "free": s["free"],
            "count": s["count"]}


def work(case):
    st = _structure(case)
    if case["op"] == "attn":
        rows = case["drafts"] * case["heads"]
        B = case["requests"]
        keys = sum(st["shared"]) + sum(st["own"])                    # each distinct row once
        return {"bytes": B * rows * (D * 2 + DV * 2 + 4) + keys * D * 2, "flops": 2.0 * (D + DV) * rows * sum(st["kv_lens"])}
    if case["op"] == "append":
        N = case["tokens"] - case["pad"]
        per_head = (D if case["absorbed"] else DR) * 2 * 2
        return {"bytes": N * (2 * D * 2 + DR * 4 + 8 + case["heads"] * per_head), "flops": N * (4 * D + case["heads"] * 3 * DR)}
    entries = copied = dropped = 0
    for p in st["parents"]:
        n = st["lens"][p]
        entries += -(-(n + case["extra"]) // PAGE)
        copied += n % PAGE
    dropped = sum(-(-n // PAGE) for n in st["lens"]) if case["beam"] else entries
    # an entry read and written with its count read and written; a dropped one read, with its count; rows both ways
    return {"bytes": entries * 16 + dropped * 12 + copied * case["layers"] * D * 2 * 2, "flops": 0}


# ---- the definition, in 64 bits ------------------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "fork":
        return None                                                  # pages are moved and counted: no computed numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        cs = s["cos_sin"].double()[s["pos"].long()]
        z = torch.complex(cs[:, :32], cs[:, 32:])

        def turn(x, z):
            pair = x.unflatten(-1, (32, 2)) if case["interleaved"] else x.unflatten(-1, (2, 32)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
            return y.flatten(-2) if case["interleaved"] else y.transpose(-1, -2).flatten(-2)

        kv, cache, q = s["kv"].double(), s["cache"].double(), s["q"].double()
        real = (s["slots"] >= 0).nonzero()[:, 0]
        c = kv[real, :DV]
        norm = c / (c.pow(2).sum(-1, keepdim=True) / DV + EPS).sqrt() * s["weight"].double()
        cache[s["slots"][real].long()] = torch.cat((norm, turn(kv[real, DV:], z[real])), -1)
        q[real, :, DV:] = turn(s["q_pe"].double()[real], z[real][:, None])
        if s["q_nope"] is not None:
            q[real, :, :DV] = s["q_nope"].double()[real]
        return {"q": q, "cache": cache}
    B, T, H, _ = s["q"].shape
    lens = s["kv_lens"].tolist()
    if 2176.0 * T * H * sum(lens) > 6e12:
        return None
    outs, lses = [], []
    for b in range(B):
        n, at = lens[b], int(s["kv_indptr"][b])
        if case["page"] == 1:
            slot = s["kv_indices"][at:at + n].long()
        else:
            slot = (s["kv_indices"][at:at + -(-n // PAGE)].long()[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()[:n]
        k = s["cache"][slot].double()
        tree = s["parent"][b].tolist()
        for t in range(T):
            seen = torch.ones(n, dtype=torch.bool, device="cuda")
            seen[n - T:] = False
            i = t
            while i >= 0:
                seen[n - T + i] = True
                i = tree[i]
            x = (s["q"][b, t].double() @ k[seen].T) * SCALE
            lse = torch.logsumexp(x, -1)
            outs.append(torch.exp(x - lse[:, None]) @ k[seen][:, :DV])
            lses.append(lse)
    return {"out": torch.stack(outs).reshape(B, T, H, DV), "lse": torch.stack(lses).reshape(B, T, H)}
