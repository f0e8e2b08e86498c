"""Seeded paged caches for the tests of the attention over them, and the
bounds that its outputs are held to."""
import numpy as np
import torch

import oracle


def make(lens, news, page, hq, hk, d, seed, plens=None, first=None, slots=None, layout="plain", device="cuda",
         garbage=float("nan"), extra_tokens=0):
    """Inputs of one call on `device`, and the same in float64 on the host.
    Places behind a sequence's end hold `garbage`, unused table entries a page
    index far outside the pool."""
    rng = np.random.default_rng(seed)
    rows = list(plens or []) + list(lens)
    need = [-(-n // page) for n in rows]
    n_pages = sum(need) + 5
    order = rng.permutation(n_pages)
    width = max(need + [1]) + 2
    table = np.full((len(rows), width), 1 << 28, np.int32)
    kv = torch.from_numpy(rng.standard_normal((2, n_pages, page, hk, d)).astype(np.float32)).bfloat16()
    live = np.zeros((n_pages, page), bool)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        j = np.arange(rows[b])
        live[table[b, j // page], j % page] = True
    ref = kv.double().numpy() * live[None, :, :, None, None]
    kv = kv.masked_fill(~torch.from_numpy(live)[None, :, :, None, None], garbage)
    q_ptr = np.concatenate([[0], np.cumsum(news)]).astype(np.int32) + extra_tokens
    T = int(q_ptr[-1]) + extra_tokens
    q = torch.from_numpy(rng.standard_normal((T, hq, d)).astype(np.float32)).bfloat16()
    np_ = len(plens or [])
    c = {"q_ptr": q_ptr, "lens": np.asarray(lens, np.int32), "table": table[np_:], "ptable": table[:np_],
         "plens": np.asarray(plens or [], np.int32), "first": np.asarray(first if first is not None else [], np.int32),
         "scale": 1.0 / np.sqrt(d), "seqs": None, "k64": ref[0], "v64": ref[1], "q64": q.double().numpy()}
    if slots is not None:        # the sequences sit in chosen rows of a larger table
        big, bl = np.full((max(slots) + 3, width), -1, np.int32), np.zeros(max(slots) + 3, np.int32)
        big[slots], bl[slots] = c["table"], c["lens"]
        c["table"], c["lens"], c["seqs"] = big, bl, np.asarray(slots, np.int32)
    if layout == "plain":
        c["k"], c["v"] = (x.contiguous().to(device) for x in kv)
    elif layout == "joined":     # keys and values of a page side by side
        x = kv.transpose(0, 1).contiguous().to(device)
        c["k"], c["v"] = x[:, 0], x[:, 1]
    elif layout == "heads":      # head-major pages, and rows wider than d
        x = torch.full((2, n_pages, hk, page, d + 8), garbage, dtype=torch.bfloat16, device=device)
        x[..., :d] = kv.permute(0, 1, 3, 2, 4).to(device)
        c["k"], c["v"] = (y[..., :d].permute(0, 2, 1, 3) for y in x)
    c["q"] = q.to(device)
    for name in ("q_ptr", "lens", "table", "ptable", "plens", "first", "seqs"):
        c["d_" + name] = None if c[name] is None else torch.from_numpy(np.ascontiguousarray(c[name])).to(device)
    return c


def reference(c, window=0, sinks=0):
    prefix = (c["ptable"], c["plens"], c["first"]) if len(c["plens"]) else None
    return oracle.oracle_paged(c["q64"], c["k64"], c["v64"], c["table"], c["lens"], c["q_ptr"], c["scale"], window, sinks,
                               c["seqs"], prefix)


def check(c, out, lse, ref):
    """Holds every row of a sequence to its rounding bound.

    u = 2^-24 (f32 half step), h = 2^-8 (bf16 half step), N keys.
    A score sums d products in f32 and is scaled: off by at most
    e = (d + 4) u scale sum|q||k|, and exp2 adds 2^-22 relative (and the two
    roundings of its argument, 2 u |s| log2 e ln 2, within another 4 u scale
    sum|q||k|).  A weight is thus off by r = e + 4 u scale sum|q||k| + 2^-22,
    doubled in the quotient with their sum; sums over N keys in f32 add N u;
    P is rounded to bf16 before its product, h each; merges of pieces and
    prefixes scale each sum once more (2^-22).  With A = sum p|v|:
      |dO| <= A (2 r + h + 2 N u + 2^-21)   and a bf16 O half a step more;
      |dlse| <= r + N u + 2^-21 + 2 u |lse|.
    """
    O, L, A, big = ref
    d, n = O.shape[2], int(max(list(c["lens"]) + [1])) + int(max(list(c["plens"]) + [0]))
    u, h = 2.0 ** -24, 2.0 ** -8
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    mine = ~np.isnan(L[0])
    o, l, O, L, A, big = o[mine], l[:, mine], O[mine], L[:, mine], A[mine], big[:, mine]
    empty = np.isneginf(L)
    assert np.array_equal(np.isneginf(l), empty)
    assert np.all(o[empty.T] == 0)
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(l[~empty]))
    r = (d + 8) * u * big + 2.0 ** -22
    bound = A * ((2 * r + 2 * n * u + 2.0 ** -21).T[:, :, None] + h)
    if out.dtype == torch.bfloat16:
        bound = bound + h * (np.abs(O) + bound)
    off = np.abs(o - O) - bound
    assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))
    ok = ~empty
    offl = np.abs(l[ok] - L[ok]) - (r[ok] + n * u + 2.0 ** -21 + 2 * u * np.abs(L[ok]))
    assert offl.size == 0 or offl.max() <= 0, offl.max()
