"""Workloads of the paged-cache operators: a verification step of drafted tokens and the pages below it.

Six calls over one paged key/value cache (16-token pages, the layouts of paged_attn_decode):

  tree     attention of each sequence's drafted tokens, a tree, over its cached context and their own ancestors
  write    the keys and values of new tokens go into the pages of their sequences
  accept   the tokens of the accepted path of a draft move up to the end of the context
  fork     rows of the block table are freed and become copies of others: whole pages shared, a partial last page copied
  compact  the used pages of a pool move to its lowest ids

A case is a dict; `listed()` names twelve, `draw(rng)` gives another of the same ranges, `prepare` makes its inputs on the
GPU, `run` is one pass, `work` what a pass cannot do without, `exact` the definition in 64 bits.  With `own` false a pass
computes the operators from elementary torch operations.
"""
import torch

own = False

PAGE = 16        # tokens of a page
X = 8            # elements of a 16-byte piece of a key
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# (query heads, key/value heads): those of the decode workloads
HEADS = [(16, 16), (16, 2), (3, 3), (32, 4), (32, 8), (4, 1), (40, 8), (64, 8)]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # four requests in their first turn, eight drafts each: latency
        {"name": "tree_first_turn", "op": "tree", "seqs": 4, "ctx": 128, "new": 8, "hq": 32, "hkv": 8, "d": 128,
         "type": "fp16", "ragged": False},
        # a full server, equal contexts of 4096, sixteen drafts each: the stream of keys and values
        {"name": "tree_batch_4096", "op": "tree", "seqs": 64, "ctx": 4096, "new": 16, "hq": 32, "hkv": 8, "d": 128,
         "type": "bf16", "ragged": False},
        # few long documents of unequal length: the keys of one sequence have to be split
        {"name": "tree_long_ragged", "op": "tree", "seqs": 3, "ctx": 131071, "new": 33, "hq": 40, "hkv": 8, "d": 128,
         "type": "bf16", "ragged": True},
        # wide trees on a large head size: 512 query rows read each key
        {"name": "tree_wide_d256", "op": "tree", "seqs": 16, "ctx": 2112, "new": 64, "hq": 32, "hkv": 4, "d": 256,
         "type": "fp16", "ragged": True},
        # a decode step of a full server: one token for each sequence
        {"name": "write_decode", "op": "write", "seqs": 256, "ctx": 64, "new": 1, "hkv": 16, "d": 128, "type": "bf16",
         "ragged": True},
        # a prefill batch of ragged prompts
        {"name": "write_prefill", "op": "write", "seqs": 12, "ctx": 0, "new": 4195, "hkv": 8, "d": 128, "type": "bf16",
         "ragged": True},
        # four requests accept up to four of eight drafts
        {"name": "accept_few", "op": "accept", "seqs": 4, "ctx": 128, "new": 8, "take": 4, "hkv": 8, "d": 128,
         "type": "fp16", "ragged": False},
        # a full server accepts paths of up to twelve of 64 drafts
        {"name": "accept_full", "op": "accept", "seqs": 256, "ctx": 1024, "new": 64, "take": 12, "hkv": 8, "d": 128,
         "type": "bf16", "ragged": True},
        # one request with four beams
        {"name": "fork_beams", "op": "fork", "forks": 4, "ctx": 276, "hkv": 8, "d": 128, "type": "bf16", "ragged": False},
        # 256 beams over long contexts: tables and counts of 66 thousand pages
        {"name": "fork_full", "op": "fork", "forks": 256, "ctx": 4100, "hkv": 2, "d": 128, "type": "bf16", "ragged": True},
        # a small pool, half used
        {"name": "compact_small", "op": "compact", "pages": 256, "rows": 8, "used": 0.5, "hkv": 8, "d": 128,
         "type": "bf16"},
        # a pool of a gigabyte, 60 % used after many requests came and went
        {"name": "compact_large", "op": "compact", "pages": 16384, "rows": 96, "used": 0.6, "hkv": 8, "d": 128,
         "type": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "write", "accept", "fork", "compact"])
    hq, hkv = rng.choice(HEADS)
    c = {"op": op, "hkv": hkv, "d": rng.choice([64, 128, 128, 256]), "type": rng.choice(["bf16", "fp16"])}
    limit = 64 * 4096 * 8 * 128  # elements of the keys of the largest listed case
    if op == "tree":
        c.update(hq=hq, seqs=_log(rng, 1, 256), new=_log(rng, 1, 64), ragged=rng.random() < 0.6)
        c["ctx"] = _log(rng, 1, max(2, min(131072, limit // (c["seqs"] * hkv * c["d"]))))
        rows = c["seqs"] * c["new"] * hq * (c["ctx"] + c["new"]) * c["d"]
        if rows > 16 * 64 * 32 * 2112 * 256:  # the operations of the widest listed case
            c["ctx"] = max(1, c["ctx"] * (16 * 64 * 32 * 2112 * 256) // rows)
    elif op == "write":
        c.update(seqs=_log(rng, 1, 256), ctx=_log(rng, 1, 512), ragged=rng.random() < 0.7)
        c["new"] = _log(rng, 1, max(1, min(4195, 12 * 4195 * 8 * 128 // (c["seqs"] * hkv * c["d"]))))
    elif op == "accept":
        c.update(seqs=_log(rng, 1, 256), new=_log(rng, 2, 64), ragged=rng.random() < 0.5, ctx=_log(rng, 1, 1024))
        c["take"] = rng.randint(1, min(12, c["new"]))
    elif op == "fork":
        c.update(forks=_log(rng, 1, 256), ctx=_log(rng, 1, 4100), hkv=rng.choice([1, 2]), d=rng.choice([64, 128]),
                 ragged=rng.random() < 0.5)
    else:
        c.update(pages=_log(rng, 64, 16384), rows=_log(rng, 1, 96), used=round(0.1 + 0.85 * rng.random(), 3),
                 hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]))
    return c


# ---------------------------------------------------------------- lengths
def _lens(case, n):
    """(context lengths, new tokens) of n sequences: the case's numbers, or ragged from a fixed pattern below them."""
    ctx, new = case["ctx"], case.get("new", 0)
    if not case.get("ragged"):
        return [ctx] * n, [new] * n
    return ([int(ctx * (1.0 - (0.618034 * i) % 1.0)) for i in range(n)],
            [max(1, int(new * (1.0 - (0.414214 * i) % 1.0))) if new else 0 for i in range(n)])


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _page_bytes(case):
    """Bytes of one page's keys, or of its values."""
    return case["hkv"] * PAGE * case["d"] * 2


def _used_rows(case):
    """Pages of each row of a pool to be compacted."""
    used = max(1, int(case["pages"] * case["used"]))
    rows = min(case["rows"], used)
    return [used // rows + (1 if i < used % rows else 0) for i in range(rows)]


def work(case):
    op, d = case["op"], case["d"]
    if op == "tree":
        ctx, new = _lens(case, case["seqs"])
        keys = sum(c + t for c, t in zip(ctx, new))
        rows = sum(new) * case["hq"]
        pairs = sum(t * (c + (t + 1) / 2) for c, t in zip(ctx, new)) * case["hq"]
        return {"bytes": keys * case["hkv"] * d * 4 + rows * d * 4 + 4 * sum(_pages(c + t) for c, t in zip(ctx, new)),
                "flops": 4 * d * pairs}
    if op == "write":
        _, new = _lens(case, case["seqs"])
        return {"bytes": sum(new) * case["hkv"] * d * 2 * 2 * 2 + 8 * case["seqs"], "flops": 0}
    if op == "accept":
        _, new = _lens(case, case["seqs"])
        moved = sum(min(1 + i % case["take"], t) for i, t in enumerate(new))
        return {"bytes": moved * case["hkv"] * d * 2 * 2 * 2 + 12 * case["seqs"], "flops": 0}
    if op == "fork":
        ctx, _ = _lens(case, case["forks"])
        part = sum(1 for c in ctx if c % PAGE)
        # copied pages; the table's entries read and written; a count taken down and one put up for each entry
        return {"bytes": 4 * part * _page_bytes(case) + sum(_pages(c) for c in ctx) * (8 + 4 + 16), "flops": 0}
    used = sum(_used_rows(case))
    moves = used * (1 - used / case["pages"])
    return {"bytes": 4 * moves * _page_bytes(case) + 8 * used + 8 * case["pages"], "flops": 0}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _caches(case, blocks, g):
    t = TYPES[case["type"]]
    k = torch.randn((blocks, case["hkv"], case["d"] // X, PAGE, X), generator=g, device="cuda", dtype=t)
    v = torch.randn((blocks, case["hkv"], case["d"], PAGE), generator=g, device="cuda", dtype=t)
    return k, v


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(pages, spare, g):
    """A block table with shuffled pages: rows of `pages`, and the blocks of its pool."""
    total = sum(pages)
    ids = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)[:total]
    width = max(1, max(pages))
    counts = _i32(pages)
    at = torch.arange(width, device="cuda", dtype=torch.int32)[None, :]
    start = (torch.cumsum(counts, 0, dtype=torch.int32) - counts)[:, None]
    live = at < counts[:, None]
    table = torch.where(live, ids[(start + at).clamp(0, max(total - 1, 0)).long()], torch.zeros_like(at))
    return table.contiguous(), total + spare


def prepare(case, seed):
    g = _gen(seed)
    op, d, t = case["op"], case["d"], TYPES[case["type"]]
    s = {"op": op}
    if op in ("tree", "write", "accept"):
        ctx, new = _lens(case, case["seqs"])
        lens = [c + n for c, n in zip(ctx, new)]
        s["table"], blocks = _tables([_pages(n) for n in lens], 16, g)
        s["k"], s["v"] = _caches(case, blocks, g)
        s["lens"] = _i32(lens)
        s["cu"] = torch.nn.functional.pad(torch.cumsum(_i32(new), 0, dtype=torch.int32), (1, 0))
        s["total"], s["widest"], s["longest"] = sum(new), max(new), max(lens)
    if op == "tree":
        s["q"] = torch.randn((s["total"], case["hq"], d), generator=g, device="cuda", dtype=t)
        # a draft hangs on one of the three before it, or on the context
        inside = torch.arange(s["total"], device="cuda") - s["cu"][:-1].long().repeat_interleave(_i32(new).long())
        back = torch.randint(1, 4, (s["total"],), generator=g, device="cuda")
        s["parents"] = (inside - back).clamp(min=-1).to(torch.int32)
    elif op == "write":
        # the two halves of one projection's output
        kv = torch.randn((s["total"], 2, case["hkv"], d), generator=g, device="cuda", dtype=t)
        s["key"], s["value"] = kv[:, 0], kv[:, 1]
    elif op == "accept":
        n, take, wide = case["seqs"], case["take"], s["widest"]
        # of each sequence's drafts an increasing choice: the smallest of random keys, in order
        order = torch.rand((n, wide), generator=g, device="cuda")
        order = torch.where(torch.arange(wide, device="cuda")[None, :] < _i32(new)[:, None], order, order + 2.0)
        some = _i32([min(1 + i % take, t_) for i, t_ in enumerate(new)])
        pick = torch.argsort(order, dim=1)[:, :take]
        pick = torch.where(torch.arange(take, device="cuda")[None, :] < some[:, None], pick, pick + wide)
        s["accepted"] = torch.sort(pick, dim=1).values.to(torch.int32).contiguous()
        s["some"] = some
    elif op == "fork":
        n = case["forks"]
        ctx, _ = _lens(case, n)
        # rows [0, n) hold sequences; rows [n, 2 n) are forks of them from the step before
        pages = [_pages(c) for c in ctx] + [1 if c % PAGE else 0 for c in ctx]
        table, blocks = _tables(pages, n + 16, g)
        mine, fresh = table[:n], table[n:, :1]
        at = torch.arange(mine.shape[1], device="cuda", dtype=torch.int32)[None, :]
        lens = _i32(ctx)
        last = (at == lens[:, None] // PAGE) & (lens[:, None] % PAGE != 0)
        s["table"] = torch.cat([mine, torch.where(last, fresh, mine)]).contiguous()
        s["lens"] = torch.cat([lens, lens]).contiguous()
        live = at < ((torch.cat([lens, lens]) + PAGE - 1) // PAGE)[:, None]
        s["refs"] = torch.bincount(s["table"][live].long(), minlength=blocks).to(torch.int32)
        s["k"], s["v"] = _caches(case, blocks, g)
        s["src"] = torch.randint(0, n, (n,), generator=g, device="cuda", dtype=torch.int32)
        s["dst"] = torch.arange(n, 2 * n, device="cuda", dtype=torch.int32)
    elif op == "compact":
        rows = _used_rows(case)
        s["table"], blocks = _tables(rows, case["pages"] - sum(rows), g)
        s["lens"] = _i32([r * PAGE - i % PAGE for i, r in enumerate(rows)])
        live = torch.arange(s["table"].shape[1], device="cuda")[None, :] < _i32(rows)[:, None]
        s["refs"] = torch.bincount(s["table"][live].long(), minlength=blocks).to(torch.int32)
        s["k"], s["v"] = _caches(case, blocks, g)
    return s


# ----------------------------------------------------------------- a pass
def run(s):
    op = s["op"]
    if own:
        import variable_length_prefill_gb300 as vlp
        if op == "tree":
            return {"out": vlp.paged_attn_tree(s["q"], s["k"], s["v"], s["table"], s["lens"], s["cu"], s["parents"])}
        if op == "write":
            vlp.paged_attn_cache_write(s["key"], s["value"], s["k"], s["v"], s["table"], s["lens"], s["cu"])
            return {"k": s["k"], "v": s["v"]}
        if op == "accept":
            lens = vlp.paged_attn_cache_accept(s["k"], s["v"], s["table"], s["lens"], s["cu"], s["accepted"], s["some"])
            return {"k": s["k"], "v": s["v"], "lens": lens}
        if op == "fork":
            vlp.paged_attn_cache_free(s["table"], s["lens"], s["refs"], s["dst"])
            vlp.paged_attn_cache_fork(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["src"], s["dst"])
            return {"k": s["k"], "v": s["v"], "table": s["table"], "lens": s["lens"], "refs": s["refs"]}
        table, refs = vlp.paged_attn_cache_compact(s["k"], s["v"], s["table"], s["lens"], s["refs"])
        return {"k": s["k"], "v": s["v"], "table": table, "refs": refs}
    return {"tree": _tree, "write": _write, "accept": _accept, "fork": _fork, "compact": _compact}[op](s)


def _twice(r):
    """Reach over twice as many steps."""
    return (r @ r).clamp_(max=1.0)


def _inside(s):
    """(sequence, index in its drafts) of each packed row."""
    row = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    return seq, row - s["cu"].long()[seq]


def _tree(s):
    q, k, v, lens, cu = s["q"], s["k"], s["v"], s["lens"].long(), s["cu"].long()
    n, wide = lens.numel(), s["widest"]
    hq, d, hkv = q.shape[1], q.shape[2], k.shape[1]
    group = hq // hkv
    seq, j = _inside(s)
    count = cu[1:] - cu[:-1]
    # who sees whom among the drafts: the closure of "hangs on", by squaring (2^6 steps reach over 64 drafts)
    sees = torch.eye(wide, device="cuda").expand(n, wide, wide).contiguous()
    p = s["parents"].long()
    sees[seq, j, p.clamp(min=0)] += (p >= 0).float()
    sees = sees.clamp_(max=1.0)
    sees = _twice(_twice(_twice(_twice(_twice(_twice(sees)))))) > 0
    # keys and values of every position of the tables, in 32 bits
    page = s["table"].long()
    keys = k[page].float().permute(0, 2, 1, 4, 3, 5).reshape(n, hkv, -1, d)
    values = v[page].float().permute(0, 2, 1, 4, 3).reshape(n, hkv, -1, d)
    at = torch.arange(keys.shape[2], device="cuda")
    values = torch.where((at[None, :] < lens[:, None])[:, None, :, None], values, 0.0)
    rows = torch.zeros((n, wide, hq, d), device="cuda")
    rows[seq, j] = q.float()
    rows = rows.view(n, wide, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, wide * group, d)
    score = torch.matmul(rows, keys.transpose(2, 3)) * (d ** -0.5)
    base = (lens - count)[:, None]
    draft = (at[None, :] - base).clamp(0, wide - 1)
    seen = torch.where((at[None, :] < base)[:, None, :], True,
                       torch.gather(sees, 2, draft[:, None, :].expand(n, wide, at.numel())))
    seen = seen & (at[None, :] < lens[:, None])[:, None, :]
    seen = seen[:, None, :, None, :].expand(n, 1, wide, group, at.numel()).reshape(n, 1, wide * group, -1)
    score = score.masked_fill_(~seen, float("-inf"))
    top = score.amax(dim=-1, keepdim=True)
    weight = score.sub_(torch.where(top.isinf(), 0.0, top)).exp_()
    total = weight.sum(dim=-1, keepdim=True)
    out = torch.matmul(weight, values) / torch.where(total > 0, total, 1.0)
    out = out.view(n, hkv, wide, group, d).permute(0, 2, 1, 3, 4).reshape(n, wide, hq, d)
    return {"out": out[seq, j].to(q.dtype)}


def _write(s):
    k, v = s["k"], s["v"]
    seq, j = _inside(s)
    cu, lens = s["cu"].long(), s["lens"].long()
    pos = (lens - (cu[1:] - cu[:-1]))[seq] + j
    page = s["table"].long()[seq, pos // PAGE]
    k[page, :, :, pos % PAGE] = s["key"].reshape(s["total"], k.shape[1], -1, X)
    v[page, :, :, pos % PAGE] = s["value"]
    return {"k": k, "v": v}


def _accept(s):
    k, v = s["k"], s["v"]
    cu, lens = s["cu"].long(), s["lens"].long()
    base = (lens - (cu[1:] - cu[:-1]))[:, None]
    m = torch.arange(s["accepted"].shape[1], device="cuda")[None, :]
    taken = m < s["some"][:, None]
    # an entry that is not taken repeats the row's first, which always is
    src = base + torch.where(taken, s["accepted"], s["accepted"][:, :1]).long()
    dst = base + torch.where(taken, m, 0)
    table = s["table"].long()
    from_page, to_page = torch.gather(table, 1, src // PAGE), torch.gather(table, 1, dst // PAGE)
    key, value = k[from_page, :, :, src % PAGE], v[from_page, :, :, src % PAGE]
    k[to_page, :, :, dst % PAGE] = key
    v[to_page, :, :, dst % PAGE] = value
    return {"k": k, "v": v, "lens": (base[:, 0] + s["some"]).to(torch.int32)}


def _fork(s):
    k, v, table, lens, refs = s["k"], s["v"], s["table"], s["lens"], s["refs"]
    src, dst = s["src"].long(), s["dst"].long()
    at = torch.arange(table.shape[1], device="cuda")[None, :]
    # free: each page of the rows is held once less
    live = at < ((lens[dst] + PAGE - 1) // PAGE)[:, None]
    old = table[dst]
    refs.index_add_(0, torch.where(live, old, 0).reshape(-1).long(), -live.reshape(-1).to(torch.int32))
    lens[dst] = 0
    # fork
    size = lens[src].long()
    part, full = size % PAGE != 0, (size // PAGE)[:, None]
    free = torch.argsort((refs > 0).to(torch.uint8), stable=True)
    fresh = free[(torch.cumsum(part, 0) - 1).clamp(min=0)].to(torch.int32)
    theirs = table[src]
    mine = torch.where(at < full, theirs, torch.where((at == full) & part[:, None], fresh[:, None], old))
    table[dst] = mine
    lens[dst] = size.to(torch.int32)
    shared = at < full
    refs.index_add_(0, torch.where(shared, theirs, 0).reshape(-1).long(), shared.reshape(-1).to(torch.int32))
    refs.index_add_(0, torch.where(part, fresh, 0).long(), part.to(torch.int32))
    last = torch.gather(theirs, 1, full.clamp(max=table.shape[1] - 1))[:, 0]
    to, last = fresh[part].long(), last[part].long()
    k[to] = k[last]
    v[to] = v[last]
    return {"k": k, "v": v, "table": table, "lens": lens, "refs": refs}


def _compact(s):
    k, v, table, refs = s["k"], s["v"], s["table"], s["refs"]
    used = refs > 0
    ids = torch.arange(refs.numel(), device="cuda")
    low = torch.nonzero(~used & (ids < used.sum()))[:, 0]          # the lowest hole
    high = torch.nonzero(used & (ids >= used.sum()))[:, 0].flip(0)  # gets the highest used page
    now = ids.to(torch.int32)
    now[high] = low.to(torch.int32)
    k[low] = k[high]
    v[low] = v[high]
    count = refs.clone()
    count[low] = refs[high]
    count[high] = 0
    live = torch.arange(table.shape[1], device="cuda")[None, :] < ((s["lens"] + PAGE - 1) // PAGE)[:, None]
    return {"k": k, "v": v, "table": torch.where(live, now[table.long()], table), "refs": count}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    k, v = s["k"].double(), s["v"].double()
    table, lens = s["table"].tolist(), s["lens"].tolist()
    if op in ("tree", "write", "accept"):
        cu = s["cu"].tolist()
    if op == "tree":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        group = case["hq"] // case["hkv"]
        parents = s["parents"].tolist()
        for i, n in enumerate(lens):
            lo, hi = cu[i], cu[i + 1]
            ids = torch.tensor(table[i][:_pages(n)], device="cuda")
            keys = k[ids].permute(1, 0, 3, 2, 4).reshape(case["hkv"], -1, case["d"])[:, :n]
            values = v[ids].permute(1, 0, 3, 2).reshape(case["hkv"], -1, case["d"])[:, :n]
            mask = torch.ones((hi - lo, n), dtype=torch.bool)
            for j in range(hi - lo):
                mask[j, n - (hi - lo):] = False
                a = j
                while a >= 0:
                    mask[j, n - (hi - lo) + a] = True
                    a = parents[lo + a]
            mask = mask.cuda()
            for h in range(case["hq"]):
                score = s["q"][lo:hi, h].double() @ keys[h // group].T / case["d"] ** 0.5
                out[lo:hi, h] = torch.softmax(score.masked_fill(~mask, float("-inf")), dim=1) @ values[h // group]
        return {"out": out}
    if op == "write":
        for i, n in enumerate(lens):
            lo, hi = cu[i], cu[i + 1]
            pos = torch.arange(n - (hi - lo), n)
            ids, at = torch.tensor(table[i])[pos // PAGE].cuda(), (pos % PAGE).cuda()
            for h in range(case["hkv"]):
                v[ids, h, :, at] = s["value"][lo:hi, h].double()
                for x in range(case["d"] // X):
                    k[ids, h, x, at] = s["key"][lo:hi, h, x * X:x * X + X].double()
        return {"k": k, "v": v}
    if op == "accept":
        accepted, some = s["accepted"].tolist(), s["some"].tolist()
        after = []
        for i, n in enumerate(lens):
            base = n - (cu[i + 1] - cu[i])
            for m in range(some[i]):  # in this order no draft is overwritten before it is read
                a, b = base + accepted[i][m], base + m
                k[table[i][b // PAGE], :, :, b % PAGE] = k[table[i][a // PAGE], :, :, a % PAGE]
                v[table[i][b // PAGE], :, :, b % PAGE] = v[table[i][a // PAGE], :, :, a % PAGE]
            after.append(base + some[i])
        return {"k": k, "v": v, "lens": _i32(after)}
    refs = s["refs"].tolist()
    if op == "fork":
        src, dst = s["src"].tolist(), s["dst"].tolist()
        for r in dst:
            for b in table[r][:_pages(lens[r])]:
                refs[b] -= 1
            lens[r] = 0
        holes = (b for b, c in enumerate(list(refs)) if c == 0)
        for a, r in zip(src, dst):
            full, rest = divmod(lens[a], PAGE)
            table[r][:full] = table[a][:full]
            for b in table[a][:full]:
                refs[b] += 1
            if rest:
                b = next(holes)
                k[b], v[b] = k[table[a][full]], v[table[a][full]]
                table[r][full], refs[b] = b, 1
            lens[r] = lens[a]
        return {"k": k, "v": v, "table": _i32(table), "lens": _i32(lens), "refs": _i32(refs)}
    live = sum(1 for c in refs if c)
    now, top = {}, len(refs) - 1
    for b in range(live):
        if refs[b] == 0:
            while refs[top] == 0:
                top -= 1
            k[b], v[b], refs[b], refs[top], now[top] = k[top], v[top], refs[top], 0, b
    table = [[now.get(b, b) if c < _pages(lens[r]) else b for c, b in enumerate(row)] for r, row in enumerate(table)]
    return {"k": k, "v": v, "table": _i32(table), "refs": _i32(refs)}
