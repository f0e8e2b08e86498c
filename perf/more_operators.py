"""Measured cases of the operators over a cache held in 8 bits, and of a beam
search's step over that cache's sequences.

  paged   attention of each sequence's newest tokens over pages in 8 bits, with
          one scale for each token and key/value head
  write   new keys and values quantised as they are written to their pages
  read    cached tokens brought back as rows of 16 bits
  beam    the best continuations over beams and vocabulary, and the beams'
          states brought into their order

``own`` False computes each in plain torch; True calls the framework.
"""
import math
import random

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
E4M3 = torch.float8_e4m3fn
TOP = {"int8": 127.0, "e4m3": 448.0}


def listed():
    return [
        # one user's chat turn, one token at a time: latency of the smallest call
        {"name": "decode one sequence", "kind": "paged", "fmt": "int8", "seqs": 1, "new": 1, "lo": 16411, "hi": 16411, "window": 1024, "sinks": 4, "page": 16, "hq": 32, "hk": 8, "d": 128},
        # a serving batch of mixed lengths with a windowed model
        {"name": "decode batch, window", "kind": "paged", "fmt": "int8", "seqs": 64, "new": 1, "lo": 509, "hi": 32768, "window": 4096, "sinks": 4, "page": 64, "hq": 32, "hk": 8, "d": 128},
        # long contexts without a window, for which a cache is held in 8 bits: the cache's whole bandwidth
        {"name": "decode batch, long", "kind": "paged", "fmt": "e4m3", "seqs": 16, "new": 1, "lo": 8191, "hi": 131072, "window": 0, "sinks": 0, "page": 128, "hq": 32, "hk": 8, "d": 128},
        # speculative tokens verified together, heads of 64 columns
        {"name": "verify batch", "kind": "paged", "fmt": "e4m3", "seqs": 48, "new": 5, "lo": 130, "hi": 16384, "window": 2048, "sinks": 1, "page": 32, "hq": 32, "hk": 8, "d": 64},
        # prompts taken in pieces over what is cached already
        {"name": "prompt pieces", "kind": "paged", "fmt": "int8", "seqs": 4, "new": 1021, "lo": 2048, "hi": 16384, "window": 4096, "sinks": 4, "page": 64, "hq": 32, "hk": 8, "d": 128},
        # one decoding step of a batch stores a token a sequence
        {"name": "step written", "kind": "write", "fmt": "e4m3", "seqs": 64, "new": 1, "lo": 64, "hi": 4096, "page": 64, "hk": 8, "d": 128},
        # a server's round of arrivals, prompts of mixed lengths
        {"name": "arrivals written", "kind": "write", "fmt": "int8", "seqs": 24, "new": 8192, "lo": 64, "hi": 8192, "page": 16, "hk": 8, "d": 128},
        # one conversation moved to another cache
        {"name": "sequence read back", "kind": "read", "fmt": "e4m3", "seqs": 1, "new": 4099, "lo": 4099, "hi": 4099, "page": 16, "hk": 8, "d": 128},
        # a whole batch moved out, two key/value heads a device
        {"name": "batch read back", "kind": "read", "fmt": "int8", "seqs": 32, "new": 32768, "lo": 509, "hi": 32768, "page": 64, "hk": 2, "d": 128},
        # a single user's beam search
        {"name": "beam step, one prompt", "kind": "beam", "dtype": "f32", "groups": 1, "beams": 4, "vocab": 32000, "history": 512, "first": False},
        # a translation server's step, an odd vocabulary, some beams finished
        {"name": "beam step, odd vocabulary", "kind": "beam", "dtype": "f32", "groups": 24, "beams": 5, "vocab": 100003, "history": 1024, "first": False},
        # a large batch, logits as the model's last product leaves them
        {"name": "beam step, large batch", "kind": "beam", "dtype": "bf16", "groups": 64, "beams": 8, "vocab": 131072, "history": 2048, "first": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["paged", "paged", "paged", "write", "read", "beam", "beam"])
    if kind == "beam":
        beams = rng.randint(1, 12)
        vocab = _log(rng, 50, 150000)
        groups = _log(rng, 1, max(1, min(96, 60_000_000 // (beams * vocab))))
        return {"kind": kind, "dtype": rng.choice(["f32", "bf16"]), "groups": groups, "beams": beams, "vocab": vocab, "history": _log(rng, 3, 2048),
                "first": rng.choice([False, False, True])}
    hq, hk, d = rng.choice([(32, 8, 128), (16, 16, 128), (16, 16, 64), (16, 2, 128), (6, 2, 64), (5, 1, 128)])
    page = rng.choice([16, 32, 64, 128, 256])
    fmt = rng.choice(["int8", "e4m3"])
    if kind == "paged":
        new = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 700)])
        seqs = _log(rng, 1, 128 if new <= 8 else 4)
        hi = _log(rng, 16 + new, min(131072, 16384 if new > 8 else (1 << 20) // seqs))
        lo = _log(rng, max(1, hi // 64), hi)
        window = rng.choice([0, _log(rng, 16, 8192)])
        return {"kind": kind, "fmt": fmt, "seqs": seqs, "new": new, "lo": lo, "hi": hi, "window": window, "sinks": rng.choice([0, 1, 4, 37]) if window else 0,
                "page": page, "hq": hq, "hk": hk, "d": d}
    hi = _log(rng, 20, 16384)
    return {"kind": kind, "fmt": fmt, "seqs": _log(rng, 1, 48), "new": rng.choice([1, _log(rng, 2, hi), hi]), "lo": max(1, hi // 40), "hi": hi, "page": page,
            "hk": hk, "d": d}


def _spread(n, lo, hi, salt):
    """n whole numbers from lo to hi, even in their logarithm, in a shuffled order of their own."""
    v = [min(hi, max(lo, int(round(lo * (hi / lo) ** ((i + 0.5) / n if n > 1 else 1.0))))) for i in range(n)]
    random.Random("%d %d %d %s" % (n, lo, hi, salt)).shuffle(v)
    return v


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _news(c):
    """Lengths of a case's sequences, and how many of each one's last tokens are the call's."""
    lens = _spread(c["seqs"], c["lo"], c["hi"], "len")
    if c["new"] == 1:
        return lens, [1] * c["seqs"]
    if c["kind"] != "paged" and c["new"] >= c["hi"]:
        return lens, lens
    return lens, [min(x, n) for x, n in zip(lens, _spread(c["seqs"], max(1, c["new"] // 2), c["new"], "new"))]


def _ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _codes(x, fmt):
    """Rows [..., d] held in 8 bits, as codes (bytes) and one scale a row: the largest
    magnitude stands at the largest code. Which code a value gets is decided in 64 bits,
    in which a value halfway between two codes stays so."""
    top = x.abs().amax(-1).float()
    t = x.double() * TOP[fmt] / top.double().clamp(min=1e-300)[..., None]
    if fmt == "int8":
        return torch.round(t).to(torch.int8), top / TOP[fmt]
    return t.float().to(E4M3).view(torch.int8), top / TOP[fmt]


def _values(codes, scales, fmt):
    """The 32-bit values that codes stand for."""
    x = codes.float() if fmt == "int8" else codes.view(E4M3).float()
    return x * scales[..., None]


def _rows(g, *shape):
    """Keys or values as a model makes them: each head of a token at its own magnitude."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=BF16)
    return x * torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=g, device="cuda")).to(BF16)


def _pool(g, rows, c):
    """Codes and scales of the sequences' tokens in pages dealt out at random, and
    their table. Places that hold no token have a code that is no number in e4m3,
    and a scale that is none, as memory never written may have."""
    page, hk, d = c["page"], c["hk"], c["d"]
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
    made = []
    for _ in range(2):
        codes = torch.empty((n_pages, page, hk, d), dtype=torch.int8, device="cuda")
        scales = torch.empty((n_pages, page, hk), device="cuda")
        step = max(1, (1 << 26) // (page * hk * d))
        for a in range(0, n_pages, step):
            b = min(n_pages, a + step)
            codes[a:b], scales[a:b] = _codes(_rows(g, b - a, page, hk, d), c["fmt"])
        codes.masked_fill_(empty[:, :, None, None], 127)
        scales.masked_fill_(empty[:, :, None], float("nan"))
        made.append((codes if c["fmt"] == "int8" else codes.view(E4M3), scales))
    return made[0] + made[1] + (table,)


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["kind"] == "beam":
        return _beams(s, c, g)
    lens, news = _news(c)
    s["k"], s["ks"], s["v"], s["vs"], s["table"] = _pool(g, lens, c)
    s["lens"] = _ints(lens)
    s["q_ptr"] = None if c["new"] == 1 else _ints(_starts(news))
    s["tokens"], s["max_new"], s["max_len"] = sum(news), max(news), max(lens)
    if c["kind"] == "paged":
        s["q"] = torch.randn((s["tokens"], c["hq"], c["d"]), generator=g, device="cuda", dtype=BF16)
    if c["kind"] == "write":
        s["k_new"], s["v_new"] = _rows(g, s["tokens"], c["hk"], c["d"]), _rows(g, s["tokens"], c["hk"], c["d"])
    return s


def _beams(s, c, g):
    """A model's logits for every beam, the beams' scores so far, which have ended
    (one in eight, but at the first step, where all beams but one of a prompt
    are still empty), and two states: the tokens chosen so far, and which tokens
    of the vocabulary a beam has used."""
    rows = c["groups"] * c["beams"]
    s["logits"] = torch.randn((rows, c["vocab"]), generator=g, device="cuda") * 2.5
    if c["dtype"] == "bf16":
        s["logits"] = s["logits"].to(BF16)
    s["scores"] = -20.0 * torch.rand((c["groups"], c["beams"]), generator=g, device="cuda")
    s["done"] = torch.rand((c["groups"], c["beams"]), generator=g, device="cuda") < 0.125
    if c["first"]:
        s["scores"][:] = -math.inf
        s["scores"][:, 0] = 0.0
        s["done"][:] = False
    s["eos"] = 2
    s["history"] = torch.randint(0, c["vocab"], (rows, c["history"]), generator=g, device="cuda", dtype=I32)
    s["used"] = torch.zeros((rows, c["vocab"]), dtype=torch.uint8, device="cuda")
    s["used"].scatter_(1, s["history"].long(), 1)
    return s


def run(state):
    s, c = state, state["case"]
    kind = c["kind"]
    if own:
        return _run_own(s, c, kind)
    if kind == "paged":
        return _paged_plain(s, c)
    if kind == "write":
        return _write_plain(s, c)
    if kind == "read":
        return _read_plain(s, c)
    return _beam_plain(s, c)


def _run_own(s, c, kind):
    import block_sparse_attention_slice_gb300 as attn
    if kind == "paged":
        return attn.attn_paged_fwd(s["q"], s["k"], s["v"], s["table"], s["lens"], 1.0 / math.sqrt(c["d"]), q_ptr=s["q_ptr"], max_q=s["max_new"],
                                   window=c["window"], sinks=c["sinks"], k_scales=s["ks"], v_scales=s["vs"])
    if kind == "write":
        attn.attn_cache_write(s["k"], s["v"], s["k_new"], s["v_new"], s["table"], s["lens"], q_ptr=s["q_ptr"], k_scales=s["ks"], v_scales=s["vs"])
        return s["k"], s["ks"], s["v"], s["vs"]
    if kind == "read":
        return attn.attn_cache_read(s["k"], s["v"], s["table"], s["lens"], s["tokens"], q_ptr=s["q_ptr"], k_scales=s["ks"], v_scales=s["vs"])
    scores, parents, tokens, done = attn.attn_beam_select(s["logits"], s["scores"], done=s["done"], eos=s["eos"])
    attn.attn_beam_reorder([s["history"], s["used"]], parents)
    return scores, parents, tokens, done, s["history"], s["used"]


# ---- plain forms -----------------------------------------------------------

def _fetch(codes, scales, fmt, table, kpos, seen):
    """Rows kpos [B, N] of each sequence in 32 bits, zero where no token is looked at."""
    page = codes.shape[1]
    at = kpos.clamp(min=0)
    slot = (at // page).clamp(max=table.shape[1] - 1)
    ids = torch.gather(table, 1, slot).long().clamp(min=0)
    return _values(codes.view(torch.int8)[ids, at % page], scales[ids, at % page], fmt).masked_fill_(~seen[:, :, None, None], 0.0)


def _paged_plain(s, c):
    q, dev, group = s["q"], s["q"].device, c["hq"] // c["hk"]
    lens = s["lens"][:, None]
    t = torch.arange(s["max_new"], device=dev)
    ptr = s["q_ptr"] if s["q_ptr"] is not None else torch.arange(len(lens) + 1, device=dev, dtype=I32)
    news = (ptr[1:] - ptr[:-1])[:, None]
    live = t[None, :] < news
    pos = lens - news + t
    if c["window"]:  # the first tokens, then all that any new token's window reaches
        first = torch.arange(c["sinks"], device=dev).expand(len(lens), -1)
        begin = (pos[:, :1] - c["window"] + 1).clamp(min=c["sinks"])
        kpos = torch.cat([first, begin + torch.arange(min(c["window"] + s["max_new"], s["max_len"]), device=dev)], 1)
    else:
        kpos = torch.arange(s["max_len"], device=dev).expand(len(lens), -1)
    inside = kpos < lens
    k, v = (_fetch(s[x], s[x + "s"], c["fmt"], s["table"], kpos, inside) for x in "kv")
    rows = q[(ptr[:-1, None] + t).clamp(max=q.shape[0] - 1)].float().unflatten(2, (c["hk"], group))
    scores = torch.einsum("bthgd,bnhd->bhgtn", rows, k) / math.sqrt(c["d"])
    far = kpos[:, None, :]
    seen = inside[:, None, :] & (far <= pos[:, :, None])
    if c["window"]:
        seen = seen & ((far < c["sinks"]) | (far > pos[:, :, None] - c["window"]))
    scores = scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1)
    o = torch.einsum("bhgtn,bnhd->bthgd", p, v)
    o = (o / total.clamp(min=1e-37).permute(0, 3, 1, 2)[..., None]).flatten(2, 3)
    lse = (top[..., 0] + torch.log(total)).permute(0, 3, 1, 2).flatten(2)
    return o[live].to(BF16), lse[live].t().contiguous()


def _places(s, c):
    """Page and row within it of each of the call's tokens."""
    dev = s["lens"].device
    ptr = s["q_ptr"] if s["q_ptr"] is not None else torch.arange(c["seqs"] + 1, device=dev, dtype=I32)
    news = (ptr[1:] - ptr[:-1]).long()
    seq = torch.repeat_interleave(torch.arange(c["seqs"], device=dev), news, output_size=s["tokens"])
    pos = s["lens"][seq] - news[seq] + torch.arange(s["tokens"], device=dev) - ptr[seq].long()
    return s["table"][seq, pos // c["page"]].long(), pos % c["page"]


def _write_plain(s, c):
    at = _places(s, c)
    k, ks = _codes(s["k_new"], c["fmt"])
    v, vs = _codes(s["v_new"], c["fmt"])
    s["k"].view(torch.int8)[at], s["ks"][at] = k, ks
    s["v"].view(torch.int8)[at], s["vs"][at] = v, vs
    return s["k"], s["ks"], s["v"], s["vs"]


def _read_plain(s, c):
    at = _places(s, c)
    return tuple(_values(s[x].view(torch.int8)[at], s[x + "s"][at], c["fmt"]).to(BF16) for x in "kv")


def _beam_plain(s, c):
    g, b, n = c["groups"], c["beams"], c["vocab"]
    x = s["logits"].double().view(g, b, n)
    top = x.amax(-1, keepdim=True)
    total = torch.exp(x - top).sum(-1, keepdim=True)
    x = x - top - torch.log(total) + s["scores"].double()[..., None]
    # a beam that has ended goes on as it is, by the token that ended it
    x = torch.where(s["done"][..., None], -math.inf, x)
    x[:, :, s["eos"]] = torch.where(s["done"], s["scores"].double(), x[:, :, s["eos"]])
    x = torch.where(torch.isnan(x), -math.inf, x).view(g, b * n)
    # the best of each prompt; equal ones by their place
    least = torch.topk(x, b, dim=1).values[:, -1:]
    group, place = torch.nonzero(x >= least, as_tuple=True)
    value = x[group, place]
    order = torch.argsort(value, descending=True, stable=True)
    order = order[torch.argsort(group[order], stable=True)]
    group, place, value = group[order], place[order], value[order]
    first = torch.searchsorted(group, torch.arange(g, device=group.device))
    at = first[:, None] + torch.arange(b, device=group.device)
    parents = (place[at] // n + torch.arange(g, device=group.device)[:, None] * b).to(I32)
    tokens = (place[at] % n).to(I32)
    done = s["done"].view(-1)[parents.long()] | (tokens == s["eos"])
    rows = parents.view(-1).long()
    s["history"].copy_(s["history"][rows])
    s["used"].copy_(s["used"][rows])
    return value[at].float(), parents, tokens, done, s["history"], s["used"]


# ---- 64 bits, from the definitions -----------------------------------------

def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["kind"] == "beam":
        best = []
        for a in range(c["groups"]):
            rows = s["logits"][a * c["beams"]:(a + 1) * c["beams"]].double()
            x = rows - torch.logsumexp(rows, -1, keepdim=True) + s["scores"][a].double()[:, None]
            x[s["done"][a]] = -math.inf
            x[s["done"][a], s["eos"]] = s["scores"][a].double()[s["done"][a]]
            best.append(torch.sort(x.flatten(), descending=True).values[:c["beams"]])
        return torch.stack(best), None, None, None, None, None
    lens, news = _news(c)
    if c["kind"] == "paged":
        parts, at = [], 0
        for b, (n, new) in enumerate(zip(lens, news)):
            i = torch.arange(n - new, n, device="cuda")[:, None]
            j = torch.arange(n, device="cuda")[None]
            seen = j <= i
            if c["window"]:
                seen = seen & ((i - j < c["window"]) | (j < c["sinks"]))
            look = torch.nonzero(seen.any(0))[:, 0]
            k, v = (_rows64(s, c, x, b, n)[look] for x in "kv")
            q = s["q"][at:at + new].double().unflatten(1, (c["hk"], -1)).permute(1, 2, 0, 3)
            x = (q @ k.permute(1, 2, 0)[:, None]) / math.sqrt(c["d"])
            x = torch.where(seen[:, look], x, -math.inf)
            lse = torch.logsumexp(x, -1)
            o = torch.exp(x - lse[..., None]) @ v.permute(1, 0, 2)[:, None]
            parts.append((o.permute(2, 0, 1, 3).flatten(1, 2), lse.flatten(0, 1)))
            at += new
        return torch.cat([o for o, _ in parts]), torch.cat([x for _, x in parts], 1)
    if c["kind"] == "read":
        return tuple(torch.cat([_rows64(s, c, x, b, n)[n - new:] for b, (n, new) in enumerate(zip(lens, news))]) for x in "kv")
    out = []
    for x in "kv":
        codes, scales = s[x].double(), s[x + "s"].double()
        at = 0
        for b, (n, new) in enumerate(zip(lens, news)):
            rows = s[x + "_new"][at:at + new].double()
            at += new
            pos = torch.arange(n - new, n, device="cuda")
            to = s["table"][b].long()[pos // c["page"]], pos % c["page"]
            top = rows.abs().max(-1).values
            scales[to] = top / TOP[c["fmt"]]
            y = rows * TOP[c["fmt"]] / top.clamp(min=1e-300)[..., None]
            # the step between neighbouring codes: 1, or by the value's power of two
            step = 1.0 if c["fmt"] == "int8" else 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            codes[to] = torch.round(y / step) * step
        out += [None if c["fmt"] == "int8" else codes, scales]
    return tuple(out)


def _rows64(s, c, x, b, n):
    """The first n cached rows of sequence b."""
    ids = s["table"][b][:-(-n // c["page"])].long()
    codes = s[x].view(torch.int8)[ids]
    codes = codes.double() if c["fmt"] == "int8" else codes.view(E4M3).double()
    return (codes * s[x + "s"][ids].double()[..., None]).flatten(0, 1)[:n]


def work(case):
    c = case
    if c["kind"] == "beam":
        rows = c["groups"] * c["beams"]
        row = c["vocab"] * (2 if c["dtype"] == "bf16" else 4)
        return {"bytes": rows * (row + 2 * (4 * c["history"] + c["vocab"]) + 24), "flops": rows * c["vocab"] * 4}
    lens, news = _news(c)
    token = c["hk"] * (c["d"] + 4)  # one token's keys, or its values, in 8 bits
    if c["kind"] != "paged":
        return {"bytes": sum(news) * 2 * (token + c["hk"] * c["d"] * 2), "flops": sum(news) * c["hk"] * c["d"] * 4}
    keys = pairs = 0
    for n, new in zip(lens, news):
        w, first = c["window"], c["sinks"]
        low = max(0, n - new - w + 1) if w else 0
        keys += n - low + min(first, low)
        pairs += sum(min(i + 1, w + min(first, max(0, i + 1 - w))) if w else i + 1 for i in range(n - new, n))
    return {"bytes": keys * 2 * token + sum(news) * c["hq"] * (4 * c["d"] + 4), "flops": pairs * c["hq"] * c["d"] * 4}
