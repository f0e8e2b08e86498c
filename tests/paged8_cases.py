"""Paged caches in 8 bits for the tests of the attention over them, and the bounds
that its outputs are held to."""
import numpy as np
import torch

import oracle
import paged_cases as P
from oracle import codes as C


def typed(codes, fmt):
    return codes if fmt == "int8" else codes.view(torch.float8_e4m3fn)


def make(fmt, lens, news, page, hq, hk, d, seed, layout="plain", spread=0.0, **kw):
    """paged_cases.make, its pages turned into codes with scales.  Places that no
    token owns hold the code of all ones below the sign (a NaN in e4m3) and a
    scale that is none.  spread: how far the magnitudes of rows lie apart (the
    standard deviation of their logarithms)."""
    c = P.make(lens, news, page, hq, hk, d, seed, device=kw.pop("device", "cuda"), garbage=float("nan"), **kw)
    dev = c["q"].device
    rng = np.random.default_rng(seed + 1)
    for x in "kv":
        rows = c[x].double().cpu().numpy()
        empty = np.isnan(rows).all(-1)
        size = np.exp(spread * rng.standard_normal(empty.shape))[..., None]
        rows = torch.from_numpy(np.where(empty[..., None], 0, rows) * size).bfloat16().double().numpy()
        codes, scales = oracle.oracle_encode(rows, fmt)
        c[x + "64"] = C.values(codes, fmt) * scales[..., None].astype(np.float64)
        codes[empty], scales[empty] = 127, np.nan
        codes, scales = torch.from_numpy(codes), torch.from_numpy(scales)
        if layout == "heads":        # head-major pages, rows of codes 16 bytes apart, scales a gap
            y = torch.full((codes.shape[0], hk, page, d + 16), 127, dtype=torch.int8)
            y[..., :d] = codes.permute(0, 2, 1, 3)
            s = torch.full((codes.shape[0], hk, page + 3), float("nan"))
            s[..., :page] = scales.permute(0, 2, 1)
            c[x], c[x + "s"] = typed(y.to(dev), fmt)[..., :d].permute(0, 2, 1, 3), s.to(dev)[..., :page].permute(0, 2, 1)
        else:
            c[x], c[x + "s"] = typed(codes.to(dev), fmt), scales.to(dev)
    return c


def check(c, out, lse, ref):
    """Holds every row of a sequence to its rounding bound: that of
    paged_cases.check (u = 2^-24, h = 2^-8, a score off by (d + 8) u of the largest
    scale sum |q||k|), and beyond it
      - 4 u of the same for the scales' products and the row's power of two, and
        2^-39 max|q| sum|k| <= 2^-39 d times it over for values of q that f16 cuts off
        (2^-40 of the row's largest, doubled for the two-sided weight);
      - h also covers the weight times the value's scale: one rounding u, then either to
        bf16 (h) or to f16 (2^-11), whose smallest step adds 2^-25 of a value's largest
        weighted code, N of them, at most: N 2^-24 max|v| in all.
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
    qtop = np.abs(c["q64"]).max() * np.abs(c["k64"]).max() * d * c["scale"]
    r = (d + 12) * u * big + 2.0 ** -22 + 2.0 ** -39 * qtop
    bound = A * ((2 * r + (2 * n + 1) * u + 2.0 ** -21).T[:, :, None] + h) + n * u * np.abs(c["v64"]).max()
    if out.dtype == torch.bfloat16:
        bound = bound + h * (np.abs(O) + bound)
    off = np.abs(o - O) - bound
    assert off.size == 0 or off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))
    ok = ~empty
    offl = np.abs(l[ok] - L[ok]) - (r[ok] + n * u + 2.0 ** -21 + 2 * u * np.abs(L[ok]))
    assert offl.size == 0 or offl.max() <= 0, offl.max()
