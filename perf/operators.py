"""Measured cases of the serving operators over a paged key/value cache, and of
the windowed mask they serve when it is trained.

  paged     attention of each sequence's newest tokens over its pages, with a
            sliding window and first tokens that stay visible
  train     the same mask over packed documents: forward and gradients
  prefix    attention of a batch whose groups of sequences share a long prefix
  fork      one beam-search reordering of the page table, with the page copies
  turnover  sequences retired, others admitted and their prompts written
  compact   sequences retired, the pool compacted, others admitted

``own`` False computes each in plain torch; True calls the framework.
"""
import math
import random

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32


def _paged(name, **kw):
    return {"name": name, "kind": "paged", **kw}


def listed():
    return [
        # one user's chat turn, one token at a time: latency of the smallest call
        _paged("decode one sequence", seqs=1, new=1, lo=16411, hi=16411, window=1024, sinks=4, page=16, hq=32, hk=8, d=128),
        # a serving batch of mixed lengths with a windowed model
        _paged("decode batch, window", seqs=64, new=1, lo=509, hi=32768, window=4096, sinks=4, page=64, hq=32, hk=8, d=128),
        # long contexts without a window: the cache's whole bandwidth
        _paged("decode batch, long", seqs=16, new=1, lo=8191, hi=131072, window=0, sinks=0, page=128, hq=32, hk=8, d=128),
        # speculative tokens verified together, one key/value head per query head
        _paged("verify batch", seqs=48, new=5, lo=130, hi=16384, window=2048, sinks=1, page=32, hq=16, hk=16, d=64),
        # prompts taken in pieces over what is cached already
        _paged("prompt pieces", seqs=4, new=1021, lo=2048, hi=16384, window=4096, sinks=4, page=64, hq=32, hk=8, d=128),
        # a training step's attention over packed documents
        {"name": "training step", "kind": "train", "tokens": 16384, "docs": 7, "window": 1024, "sinks": 4, "h": 16, "d": 128},
        # a small system prompt in front of a small batch
        {"name": "prefix, small batch", "kind": "prefix", "groups": 1, "seqs": 16, "new": 1, "prefix": 2048, "suffix": 256, "page": 16, "hq": 32, "hk": 8, "d": 128},
        # many samples drawn from one long document
        {"name": "prefix, one document", "kind": "prefix", "groups": 1, "seqs": 256, "new": 1, "prefix": 32768, "suffix": 1024, "page": 64, "hq": 32, "hk": 8, "d": 128},
        # several system prompts in one batch, ragged
        {"name": "prefix, several", "kind": "prefix", "groups": 4, "seqs": 50, "new": 2, "prefix": 16384, "suffix": 700, "page": 32, "hq": 16, "hk": 16, "d": 64},
        # a beam search's step
        {"name": "beam reordering", "kind": "fork", "prompts": 8, "beams": 4, "lo": 100, "hi": 2048, "page": 16, "pools": 4, "hk": 8, "d": 128},
        # a server's round of arrivals, page by page
        {"name": "arrivals", "kind": "turnover", "seqs": 64, "lo": 64, "hi": 8192, "page": 16, "pools": 2, "hk": 8, "d": 128},
        # a fragmented pool of several layers
        {"name": "compaction", "kind": "compact", "seqs": 96, "lo": 512, "hi": 16384, "page": 64, "pools": 4, "hk": 8, "d": 128},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["paged", "paged", "train", "prefix", "prefix", "fork", "turnover", "compact"])
    hq, hk, d = rng.choice([(32, 8, 128), (16, 16, 128), (16, 16, 64), (16, 2, 128), (6, 2, 64), (5, 1, 128)])
    page = rng.choice([16, 32, 64, 128, 256])
    if kind == "paged":
        new = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 700)])
        seqs = _log(rng, 1, 128 if new <= 8 else 4)
        hi = _log(rng, 16 + new, min(131072, 16384 if new > 8 else (1 << 20) // seqs))
        lo = _log(rng, max(1, hi // 64), hi)
        window = rng.choice([0, _log(rng, 16, 8192)])
        return {"kind": kind, "seqs": seqs, "new": new, "lo": lo, "hi": hi, "window": window, "sinks": rng.choice([0, 1, 4, 37]) if window else 0,
                "page": page, "hq": hq, "hk": hk, "d": d}
    if kind == "train":
        return {"kind": kind, "tokens": _log(rng, 200, 16384), "docs": rng.randint(1, 7), "window": _log(rng, 16, 1024), "sinks": rng.choice([0, 1, 4, 64]),
                "h": rng.choice([1, 4, 16]), "d": rng.choice([64, 128])}
    if kind == "prefix":
        seqs = _log(rng, 2, 200)
        return {"kind": kind, "groups": rng.randint(1, min(seqs, 5)), "seqs": seqs, "new": rng.choice([1, 1, 3]), "prefix": _log(rng, 100, 24000),
                "suffix": _log(rng, 3, 900), "page": page, "hq": hq, "hk": hk, "d": d}
    hi = _log(rng, 40, 8192)
    if kind == "fork":
        return {"kind": kind, "prompts": _log(rng, 1, 32), "beams": rng.randint(2, 6), "lo": max(1, hi // 9), "hi": min(hi, 2500), "page": page,
                "pools": rng.choice([1, 2, 6]), "hk": hk, "d": d}
    return {"kind": kind, "seqs": _log(rng, 4, 90), "lo": max(1, hi // 30), "hi": hi, "page": page, "pools": 2 if kind == "turnover" else rng.choice([2, 4]), "hk": hk, "d": d}


def _spread(n, lo, hi, salt):
    """n whole numbers from lo to hi, even in their logarithm, in a shuffled order of their own."""
    v = [_at(lo, hi, (i + 0.5) / n if n > 1 else 1.0) for i in range(n)]
    random.Random("%d %d %d %s" % (n, lo, hi, salt)).shuffle(v)
    return v


def _at(lo, hi, x):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** x))))


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _news(c):
    """New tokens of each sequence of a paged case, at most its length."""
    lens = _spread(c["seqs"], c["lo"], c["hi"], "len")
    return lens, [min(x, n) for x, n in zip(lens, _spread(c["seqs"], max(1, c["new"] // 2), c["new"], "new"))] if c["new"] > 1 else [1] * c["seqs"]


def _ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _pool(g, rows, page, hk, d):
    """Keys and values of the sequences' tokens in pages dealt out at random, and
    their table. Places that hold no token are NaN, as memory never written may be."""
    need = [-(-n // page) for n in rows]
    n_pages = sum(need) + 7
    order = torch.randperm(n_pages, generator=g, device="cuda").to(I32)
    table = torch.full((len(rows), max(max(need), 1)), -1, dtype=I32, device="cuda")
    filled = torch.zeros(n_pages, dtype=torch.int64, device="cuda")
    at = 0
    for b, n in enumerate(need):
        ids = order[at:at + n]
        at += n
        table[b, :n] = ids
        filled[ids.long()] = page
        if n:
            filled[ids[-1].long()] = rows[b] - (n - 1) * page
    empty = torch.arange(page, device="cuda")[None, :] >= filled[:, None]
    pools = []
    for _ in range(2):
        x = torch.randn((n_pages, page, hk, d), generator=g, device="cuda", dtype=BF16)
        pools.append(x.masked_fill_(empty[:, :, None, None], float("nan")))
    return pools[0], pools[1], table


def _tables(c):
    """Page tables of the page-moving cases on the host: rows, lengths, pages used."""
    page = c["page"]
    if c["kind"] == "fork":
        lens = _spread(c["prompts"], c["lo"], c["hi"], "len")
        rows, at = [], 0
        for n in lens:
            full, part = n // page, n % page > 0
            shared = list(range(at, at + full))
            at += full
            for _ in range(c["beams"]):
                rows.append(shared + ([at] if part else []))
                at += part
        return rows, [n for n in lens for _ in range(c["beams"])], at, at + len(rows) + 3
    lens = _spread(c["seqs"], c["lo"], c["hi"], "len")
    rows, at = [], 0
    for n in lens:
        need = -(-n // page)
        rows.append(list(range(at, at + need)))
        at += need
    return rows, lens, at, at + max(need for need in map(len, rows)) + 3


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=BF16)  # noqa: E731
    if c["kind"] == "train":
        s["lengths"] = _docs(c)
        s["q"], s["k"], s["v"], s["dout"] = (rand(c["tokens"], c["h"], c["d"]) for _ in range(4))
        return s
    if c["kind"] == "paged":
        lens, news = _news(c)
        s["k"], s["v"], s["table"] = _pool(g, lens, c["page"], c["hk"], c["d"])
        s["lens"] = _ints(lens)
        s["q_ptr"] = None if c["new"] == 1 else _ints(_starts(news))
        s["max_new"], s["max_len"] = max(news), max(lens)
        s["q"] = rand(sum(news), c["hq"], c["d"])
        return s
    if c["kind"] == "prefix":
        plens, lens, news, first = _groups(c)
        s["k"], s["v"], table = _pool(g, plens + lens, c["page"], c["hk"], c["d"])
        width = lambda v: max(1, max(-(-n // c["page"]) for n in v))  # noqa: E731
        s["ptable"], s["plens"] = table[:len(plens), :width(plens)].contiguous(), _ints(plens)
        s["table"], s["lens"] = table[len(plens):, :width(lens)].contiguous(), _ints(lens)
        s["group_ptr"] = _ints(first)
        s["q_ptr"] = None if c["new"] == 1 else _ints(_starts(news))
        s["max_new"], s["max_len"], s["max_prefix"] = max(news), max(lens), max(plens)
        starts = _starts(news)
        s["max_rows"] = max(starts[first[i + 1]] - starts[first[i]] for i in range(len(plens)))
        s["q"] = rand(sum(news), c["hq"], c["d"])
        return s
    rows, lens, used, n_pages = _tables(c)
    width = max(map(len, rows)) + 1
    s["table"] = _ints([r + [-1] * (width - len(r)) for r in rows])
    s["lens"] = _ints(lens)
    refs = [0] * n_pages
    for r in rows:
        for p in r:
            refs[p] += 1
    s["refs"] = _ints(refs)
    s["pools"] = [rand(n_pages, c["page"], c["hk"], c["d"]) for _ in range(c["pools"])]
    s["step"] = 0
    if c["kind"] == "fork":
        pick = torch.randint(0, c["beams"], (len(rows),), generator=g, device="cuda", dtype=I32)
        s["dst"] = torch.arange(len(rows), dtype=I32, device="cuda")
        s["src"] = s["dst"] - s["dst"] % c["beams"] + pick
        return s
    # a quarter of the sequences at a time: which, their lengths, their first tokens
    s["quarters"] = []
    for i in range(4):
        ids = list(range(i, c["seqs"], 4))
        s["quarters"].append((_ints(ids), _ints([lens[b] for b in ids]), _ints(_starts([lens[b] for b in ids]))))
    if c["kind"] == "turnover":
        most = max(sum(lens[b] for b in range(i, c["seqs"], 4)) for i in range(4))
        s["k_new"], s["v_new"] = rand(most, c["hk"], c["d"]), rand(most, c["hk"], c["d"])
    return s


def _docs(c):
    lens = _spread(c["docs"], 1 + c["tokens"] // (4 * c["docs"]), 1 + c["tokens"] // c["docs"], "doc")
    lens[-1] += c["tokens"] - sum(lens)
    return lens


def _groups(c):
    plens = _spread(c["groups"], max(1, c["prefix"] // 8), c["prefix"], "prefix")
    lens = _spread(c["seqs"], max(1, c["suffix"] // 100), c["suffix"], "len")
    news = [min(n, c["new"]) for n in lens]
    first = [i * c["seqs"] // c["groups"] for i in range(c["groups"] + 1)]
    return plens, lens, news, first


def run(state):
    s, c = state, state["case"]
    kind = c["kind"]
    if own:
        return _run_own(s, c, kind)
    if kind == "paged":
        return _paged_plain(s, c)
    if kind == "train":
        return _train_plain(s, c)
    if kind == "prefix":
        return _prefix_plain(s, c)
    return _pages_plain(s, c, kind)


def _run_own(s, c, kind):
    import block_sparse_attention_slice_gb300 as attn
    scale = 1.0 / math.sqrt(c["d"])
    if kind == "paged":
        return attn.attn_paged_fwd(s["q"], s["k"], s["v"], s["table"], s["lens"], scale, q_ptr=s["q_ptr"], max_q=s["max_new"],
                                   window=c["window"], sinks=c["sinks"])
    if kind == "train":
        n = c["tokens"]
        tiles = attn.attn_build_tiles(attn.attn_slices_from_windows(s["lengths"], c["window"], c["sinks"]), n, n)
        out, lse = attn.attn_fwd(s["q"], s["k"], s["v"], tiles, scale)
        return (out, lse) + attn.attn_bwd(s["q"], s["k"], s["v"], out, s["dout"], lse, tiles, scale, grad_dtype=BF16)
    if kind == "prefix":
        return attn.attn_prefix_fwd(s["q"], s["k"], s["v"], s["ptable"], s["plens"], s["group_ptr"], s["table"], s["lens"], scale,
                                    q_ptr=s["q_ptr"], max_q=s["max_new"])
    table, lens, refs, page = s["table"], s["lens"], s["refs"], c["page"]
    if kind == "fork":
        copies = attn.attn_cache_fork(table, lens, refs, s["src"], s["dst"], page)
        attn.attn_cache_copy_pages(s["pools"], copies)
        return table, lens, refs, s["pools"]
    ids, counts, starts = s["quarters"][s["step"] % 4]
    s["step"] += 1
    attn.attn_cache_free(table, lens, refs, ids, page)
    if kind == "compact":
        attn.attn_cache_copy_pages(s["pools"], attn.attn_cache_compact(table, lens, refs, page))
    attn.attn_cache_extend(table, lens, refs, ids, counts, page)
    if kind == "turnover":
        attn.attn_cache_write(s["pools"][0], s["pools"][1], s["k_new"], s["v_new"], table, lens, q_ptr=starts, seqs=ids)
    return table, lens, refs, s["pools"]


# ---- plain forms -----------------------------------------------------------

def _fetch(pages, table, kpos, seen):
    """Rows kpos [B, N] of each sequence in 32 bits, zero where no token is looked at."""
    page = pages.shape[1]
    at = kpos.clamp(min=0)
    slot = (at // page).clamp(max=table.shape[1] - 1)
    ids = torch.gather(table, 1, slot).long().clamp(min=0)
    return pages[ids, at % page].float().masked_fill_(~seen[:, :, None, None], 0.0)


def _padded(s, c, device):
    """Index of each sequence's new tokens [B, T] in q, and which exist."""
    n = s["lens"].shape[0]
    t = torch.arange(s["max_new"], device=device)
    ptr = s["q_ptr"] if s["q_ptr"] is not None else torch.arange(n + 1, device=device, dtype=I32)
    live = t[None, :] < (ptr[1:] - ptr[:-1])[:, None]
    at = (ptr[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
    pos = (s["lens"] - (ptr[1:] - ptr[:-1]))[:, None] + t
    return at, live, pos


def _softmax(scores, seen):
    """exp(scores - max), their sums and the max over the last axis; all zero where nothing is seen."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    return p, p.sum(-1), top[..., 0]


def _paged_plain(s, c):
    q, dev, group = s["q"], s["q"].device, c["hq"] // c["hk"]
    at, live, pos = _padded(s, c, dev)
    lens = s["lens"][:, None]
    if c["window"]:  # the first tokens, then all that any new token's window reaches
        first = torch.arange(c["sinks"], device=dev).expand(len(lens), -1)
        begin = (pos[:, :1] - c["window"] + 1).clamp(min=c["sinks"])
        kpos = torch.cat([first, begin + torch.arange(min(c["window"] + s["max_new"], s["max_len"]), device=dev)], 1)
    else:
        kpos = torch.arange(s["max_len"], device=dev).expand(len(lens), -1)
    inside = kpos < lens
    k, v = _fetch(s["k"], s["table"], kpos, inside), _fetch(s["v"], s["table"], kpos, inside)
    rows = q[at].float().unflatten(2, (c["hk"], group))
    scores = torch.einsum("bthgd,bnhd->bhgtn", rows, k) / math.sqrt(c["d"])
    far = kpos[:, None, :]
    seen = inside[:, None, :] & (far <= pos[:, :, None])
    if c["window"]:
        seen = seen & ((far < c["sinks"]) | (far > pos[:, :, None] - c["window"]))
    p, total, top = _softmax(scores, seen[:, None, None])
    o = torch.einsum("bhgtn,bnhd->bthgd", p, v)
    o = (o / total.clamp(min=1e-37).permute(0, 3, 1, 2)[..., None]).flatten(2, 3)
    lse = (top + torch.log(total)).permute(0, 3, 1, 2).flatten(2)
    return o[live].to(BF16), lse[live].t().contiguous()


def _train_plain(s, c):
    """Queries in blocks of `window`; each block meets itself, the block before and the document's first tokens."""
    n, w, h, d, scale = c["tokens"], c["window"], c["h"], c["d"], 1.0 / math.sqrt(c["d"])
    dev = s["q"].device
    blocks = -(-n // w)
    lengths = torch.tensor(s["lengths"], device=dev)
    doc = torch.repeat_interleave(torch.arange(len(lengths), device=dev), lengths)
    start = (torch.cumsum(lengths, 0) - lengths)[doc]
    qpos = torch.arange(blocks * w, device=dev).view(blocks, w)
    kpos = torch.cat([qpos - w, qpos], 1)
    inside = lambda x: x.clamp(0, n - 1)  # noqa: E731
    near = (qpos < n)[:, :, None] & (kpos >= 0)[:, None] & (kpos[:, None] <= qpos[:, :, None]) & (kpos[:, None] > qpos[:, :, None] - w) & (doc[inside(kpos)][:, None] == doc[inside(qpos)][:, :, None])
    q, k, v, do = (x.float().permute(1, 0, 2) for x in (s["q"], s["k"], s["v"], s["dout"]))
    zero = qpos >= n
    qb, dob = (x[:, inside(qpos)].masked_fill(zero[None, :, :, None], 0.0) for x in (q, do))
    kb, vb = k[:, inside(kpos)], v[:, inside(kpos)]
    # first tokens of every document [docs * sinks], seen where the window no longer reaches them
    fpos = ((torch.cumsum(lengths, 0) - lengths)[:, None] + torch.arange(c["sinks"], device=dev)).flatten()
    fok = (torch.arange(c["sinks"], device=dev) < lengths[:, None]).flatten()
    fdoc = torch.arange(len(lengths), device=dev).repeat_interleave(c["sinks"])
    kf, vf = k[:, inside(fpos)], v[:, inside(fpos)]
    far = fok & (fdoc == doc[inside(qpos)][:, :, None]) & (fpos <= (qpos - w)[:, :, None]) & (qpos < n)[:, :, None]
    scores = torch.cat([qb @ kb.transpose(-1, -2), torch.einsum("hbqd,hfd->hbqf", qb, kf)], -1) * scale
    p, total, top = _softmax(scores, torch.cat([near, far], -1))
    p = p / total.clamp(min=1e-37)[..., None]
    del scores
    m = 2 * w
    out = (p[..., :m] @ vb + torch.einsum("hbqf,hfd->hbqd", p[..., m:], vf))
    lse = (top + torch.log(total)).flatten(1)[:, :n]
    # gradients, with the rounded output that a training step keeps
    kept = out.to(BF16).float()
    delta = (dob * kept).sum(-1, keepdim=True)
    dp = torch.cat([dob @ vb.transpose(-1, -2), torch.einsum("hbqd,hfd->hbqf", dob, vf)], -1)
    ds = p * (dp - delta) * scale
    del dp
    dq = ds[..., :m] @ kb + torch.einsum("hbqf,hfd->hbqd", ds[..., m:], kf)
    to = inside(kpos).flatten()

    def back(x, rows):
        g = torch.zeros((h, n, d), device=dev)
        g.index_add_(1, to, (x[..., :m].transpose(-1, -2) @ rows).flatten(1, 2))
        return g.index_add_(1, inside(fpos), torch.einsum("hbqf,hbqd->hfd", x[..., m:], rows))

    whole = lambda x: x.flatten(1, 2)[:, :n].permute(1, 0, 2).to(BF16)  # noqa: E731
    turned = lambda x: x.permute(1, 0, 2).to(BF16)  # noqa: E731
    return whole(out), lse.contiguous(), whole(dq), turned(back(ds, qb)), turned(back(p, dob))


def _prefix_plain(s, c):
    q, dev, group, scale = s["q"], s["q"].device, c["hq"] // c["hk"], 1.0 / math.sqrt(c["d"])
    at, live, pos = _padded(s, c, dev)
    # the prefix: all rows of a group against it at once
    ptr = s["q_ptr"] if s["q_ptr"] is not None else torch.arange(len(s["lens"]) + 1, device=dev, dtype=I32)
    bounds = ptr[s["group_ptr"].long()]
    tok = bounds[:-1, None] + torch.arange(s["max_rows"], device=dev)
    held = tok < bounds[1:, None]
    tok = tok.clamp(max=q.shape[0] - 1)
    kpos = torch.arange(s["max_prefix"], device=dev).expand(len(bounds) - 1, -1)
    inside = kpos < s["plens"][:, None]
    rows = q[tok].float().unflatten(2, (c["hk"], group))
    scores = torch.einsum("bthgd,bnhd->bhgtn", rows, _fetch(s["k"], s["ptable"], kpos, inside)) * scale
    p, ptotal, ptop = _softmax(scores, inside[:, None, None, None])
    po = torch.einsum("bhgtn,bnhd->bthgd", p, _fetch(s["v"], s["ptable"], kpos, inside))
    flat = lambda x, keep: x.permute(0, 3, 1, 2)[keep]  # noqa: E731
    ptotal, ptop, po = flat(ptotal, held), flat(ptop, held), po[held]
    # what follows it, each sequence on its own
    kpos = torch.arange(s["max_len"], device=dev).expand(len(pos), -1)
    inside = kpos < s["lens"][:, None]
    rows = q[at].float().unflatten(2, (c["hk"], group))
    scores = torch.einsum("bthgd,bnhd->bhgtn", rows, _fetch(s["k"], s["table"], kpos, inside)) * scale
    p, total, top = _softmax(scores, (inside[:, None, :] & (kpos[:, None, :] <= pos[:, :, None]))[:, None, None])
    o = torch.einsum("bhgtn,bnhd->bthgd", p, _fetch(s["v"], s["table"], kpos, inside))
    total, top, o = flat(total, live), flat(top, live), o[live]
    # both summaries brought to the larger maximum
    big = torch.maximum(top, ptop)
    a, b = torch.exp(ptop - big), torch.exp(top - big)
    both = a * ptotal + b * total
    o = (a[..., None] * po + b[..., None] * o) / both[..., None]
    return o.flatten(1, 2).to(BF16), (big + torch.log(both)).flatten(1).t().contiguous()


def _pages_plain(s, c, kind):
    table, lens, refs, page = s["table"], s["lens"], s["refs"], c["page"]
    if kind == "fork":
        src, dst = s["src"].long(), s["dst"].long()
        n, rows = len(src), table[src]
        full, part = lens[src].long() // page, lens[src] % page > 0
        replaced = torch.zeros(len(lens), dtype=torch.bool, device=lens.device)
        replaced[dst] = True
        order = torch.arange(n, device=lens.device)
        first = torch.full((len(lens),), n, device=lens.device).scatter_reduce(0, src, order, "amin")[src] == order
        copied = part & ~(replaced[src] & first)
        fresh = torch.nonzero(refs == 0)[:int(copied.sum()), 0]
        slots = torch.arange(table.shape[1], device=lens.device)
        held = (slots < (full + part)[:, None]) & (rows >= 0)
        tail = torch.nonzero(copied)[:, 0]
        old = rows[tail, full[tail]].long()
        rows = torch.where(held, rows, -1)
        rows[tail, full[tail]] = fresh.to(I32)
        gone = table[dst]
        ones = torch.ones_like(refs)
        refs.index_add_(0, rows[rows >= 0].long(), ones[:1].expand(int((rows >= 0).sum())))
        refs.index_add_(0, gone[gone >= 0].long(), -ones[:1].expand(int((gone >= 0).sum())))
        lens[dst] = lens[src]
        table[dst] = rows
        for x in s["pools"]:
            x[fresh] = x[old]
        return table, lens, refs, s["pools"]
    ids, counts, starts = s["quarters"][s["step"] % 4]
    s["step"] += 1
    ids = ids.long()
    gone = table[ids]
    gone = gone[gone >= 0].long()
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=I32))
    table[ids], lens[ids] = -1, 0
    if kind == "compact":
        used = refs > 0
        n = int(used.sum())
        high, low = torch.nonzero(used[n:])[:, 0] + n, torch.nonzero(~used[:n])[:, 0]
        moved = torch.arange(len(refs), dtype=I32, device=refs.device)
        moved[high] = low.to(I32)
        table.copy_(torch.where(table >= 0, moved[table.clamp(min=0).long()], table))
        refs[low], refs[high] = refs[high], 0
        for x in s["pools"]:
            x[low] = x[high]
    have, want = -(-lens[ids].long() // page), -(-(lens[ids] + counts).long() // page)
    need = want - have
    owner = torch.repeat_interleave(torch.arange(len(ids), device=ids.device), need)
    slot = have[owner] + torch.arange(len(owner), device=ids.device) - (torch.cumsum(need, 0) - need)[owner]
    fresh = torch.nonzero(refs == 0)[:len(owner), 0]
    table[ids[owner], slot] = fresh.to(I32)
    refs[fresh] = 1
    lens[ids] += counts
    if kind == "turnover":
        news = (starts[1:] - starts[:-1]).long()
        seq = torch.repeat_interleave(torch.arange(len(ids), device=ids.device), news)
        pos = lens[ids][seq] - news[seq] + torch.arange(len(seq), device=ids.device) - starts[seq].long()
        at = table[ids[seq], pos // page].long()
        s["pools"][0][at, pos % page] = s["k_new"][:len(seq)]
        s["pools"][1][at, pos % page] = s["v_new"][:len(seq)]
    return table, lens, refs, s["pools"]


# ---- 64 bits, from the definitions -----------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    scale = 1.0 / math.sqrt(c["d"])
    if c["kind"] == "paged":
        lens, news = _news(c)
        parts, at = [], 0
        for b, (n, new) in enumerate(zip(lens, news)):
            i = torch.arange(n - new, n, device="cuda")[:, None]
            j = torch.arange(n, device="cuda")[None]
            seen = j <= i
            if c["window"]:
                seen = seen & ((i - j < c["window"]) | (j < c["sinks"]))
            look = torch.nonzero(seen.any(0))[:, 0]
            k, v = (_rows64(s[x], s["table"][b], n)[look] for x in "kv")
            parts.append(_attend64(s["q"][at:at + new], k, v, seen[:, look], scale))
            at += new
        return torch.cat([o for o, _ in parts]), torch.cat([x for _, x in parts], 1)
    if c["kind"] == "prefix":
        plens, lens, news, first = _groups(c)
        parts, at = [], 0
        for g, m in enumerate(plens):
            pk, pv = (_rows64(s[x], s["ptable"][g], m) for x in "kv")
            for b in range(first[g], first[g + 1]):
                n, new = lens[b], news[b]
                seen = torch.arange(m + n, device="cuda")[None] <= m + torch.arange(n - new, n, device="cuda")[:, None]
                k, v = (torch.cat([x, _rows64(s[y], s["table"][b], n)]) for x, y in ((pk, "k"), (pv, "v")))
                parts.append(_attend64(s["q"][at:at + new], k, v, seen, scale))
                at += new
        return torch.cat([o for o, _ in parts]), torch.cat([x for _, x in parts], 1)
    if c["kind"] == "train":
        return _train64(s, c, scale)
    return _pages64(s, c)


def _rows64(pages, row, n):
    page = pages.shape[1]
    return pages[row[:-(-n // page)].long()].flatten(0, 1)[:n].double()


def _attend64(q, k, v, seen, scale):
    hk = k.shape[1]
    q = q.double().unflatten(1, (hk, -1)).permute(1, 2, 0, 3)
    x = (q @ k.permute(1, 2, 0)[:, None]) * scale
    x = torch.where(seen, x, -math.inf)
    lse = torch.logsumexp(x, -1)
    o = torch.exp(x - lse[..., None]) @ v.permute(1, 0, 2)[:, None]
    return o.permute(2, 0, 1, 3).flatten(1, 2), lse.flatten(0, 1)


def _train64(s, c, scale):
    q, k, v, do = (s[x].double().permute(1, 0, 2) for x in ("q", "k", "v", "dout"))
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=F64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    begin = 0
    for n in s["lengths"]:
        for a in range(0, n, 512):
            b = min(n, a + 512)
            lo = max(0, a - c["window"] + 1)
            j = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), torch.arange(lo, b, device="cuda")])
            i = torch.arange(a, b, device="cuda")[:, None]
            seen = (j <= i) & ((j < c["sinks"]) | (i - j < c["window"]))
            rows, cols = slice(begin + a, begin + b), begin + j
            x = torch.where(seen, q[:, rows] @ k[:, cols].transpose(1, 2) * scale, -math.inf)
            lse[:, rows] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[:, rows, None])
            out[:, rows] = p @ v[:, cols]
            ds = p * (do[:, rows] @ v[:, cols].transpose(1, 2) - (do[:, rows] * out[:, rows]).sum(-1, keepdim=True)) * scale
            dq[:, rows] = ds @ k[:, cols]
            dk.index_add_(1, cols, ds.transpose(1, 2) @ q[:, rows])
            dv.index_add_(1, cols, p.transpose(1, 2) @ do[:, rows])
        begin += n
    turned = lambda x: x.permute(1, 0, 2)  # noqa: E731
    return turned(out), lse, turned(dq), turned(dk), turned(dv)


def _pages64(s, c):
    """The pages after one pass, followed one by one on the host; the whole numbers need no other value."""
    page, lens = c["page"], s["lens"].tolist()
    rows = [[p for p in r if p >= 0] for r in s["table"].tolist()]
    refs = s["refs"].tolist()
    moves = []
    if c["kind"] == "fork":
        src, dst = s["src"].tolist(), s["dst"].tolist()
        free = iter([p for p, r in enumerate(refs) if r == 0])
        taken = set()
        for a in src:
            if lens[a] % page and (a not in dst or a in taken):
                moves.append((rows[a][lens[a] // page], next(free)))
            taken.add(a)
        return None, None, None, _moved(s["pools"], moves)
    ids, counts, _ = s["quarters"][0]
    for b in ids.tolist():
        for p in rows[b]:
            refs[p] -= 1
        rows[b] = []
    if c["kind"] == "compact":
        n = sum(r > 0 for r in refs)
        moves = list(zip([p for p in range(n, len(refs)) if refs[p] > 0], [p for p in range(n) if refs[p] == 0]))
        return None, None, None, _moved(s["pools"], moves)
    free = iter([p for p, r in enumerate(refs) if r == 0])
    at = 0
    pools = [x.double() for x in s["pools"]]
    for n in counts.tolist():
        for first in range(0, n, page):
            m, p = min(page, n - first), next(free)
            for x, new in zip(pools, (s["k_new"], s["v_new"])):
                x[p, :m] = new[at:at + m].double()
            at += m
    return None, None, None, pools


def _moved(pools, moves):
    pools = [x.double() for x in pools]
    if moves:
        a, b = (torch.tensor(x, device="cuda") for x in zip(*moves))
        for x in pools:
            x[b] = x[a]
    return pools


def _visible(c, n, new):
    """Keys that one sequence's new tokens have to read, and the pairs they form."""
    if not c["window"]:
        return n, new * n - new * (new - 1) // 2
    low = max(0, n - new - c["window"] + 1)
    pairs = sum(min(i + 1, c["window"] + min(c["sinks"], max(0, i + 1 - c["window"]))) for i in range(n - new, n))
    return n - low + min(c["sinks"], low), pairs


def work(case):
    c = case
    if c["kind"] == "paged":
        seen = [_visible(c, n, new) for n, new in zip(*_news(c))]
        rows = sum(_news(c)[1])
        return {"bytes": sum(k for k, _ in seen) * c["hk"] * c["d"] * 4 + rows * c["hq"] * (4 * c["d"] + 4), "flops": sum(p for _, p in seen) * c["hq"] * c["d"] * 4}
    if c["kind"] == "train":
        pairs = sum(_visible(c, n, n)[1] for n in _docs(c))
        return {"bytes": c["tokens"] * c["h"] * (8 * c["d"] * 2 + 4), "flops": pairs * c["h"] * c["d"] * 14}
    if c["kind"] == "prefix":
        plens, lens, news, first = _groups(c)
        pairs = sum(sum(news[first[g]:first[g + 1]]) * m for g, m in enumerate(plens)) + sum(m * n - m * (m - 1) // 2 for n, m in zip(lens, news))
        return {"bytes": (sum(plens) + sum(lens)) * c["hk"] * c["d"] * 4 + sum(news) * c["hq"] * (4 * c["d"] + 4), "flops": pairs * c["hq"] * c["d"] * 4}
    rows, lens, used, n_pages = _tables(c)
    row = c["hk"] * c["d"] * 2 * c["pools"]
    if c["kind"] == "fork":  # at most one partial page a beam is copied, all but one of each source's
        parts = sum(1 for n in lens if n % c["page"]) * (c["beams"] - 1) // c["beams"]
        return {"bytes": 2 * parts * c["page"] * row + 8 * sum(map(len, rows)) + 4 * n_pages, "flops": 0}
    out = sum(lens) / 4
    table = 8 * sum(map(len, rows)) / 4 + 8 * n_pages
    return {"bytes": 2 * out * row + table, "flops": 0}
