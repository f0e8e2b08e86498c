"""A cache in 8 bits: what is written and read back against the oracle, code for
code, and the attention over it against float64."""
import numpy as np
import pytest
import torch

import oracle
import paged8_cases as P8
import paged_cases as P
from oracle import codes as C
from block_sparse_attention_slice_gb300 import (attn_beam_reorder, attn_beam_select, attn_cache_copy_pages, attn_cache_extend, attn_cache_fork,
                                                attn_cache_read, attn_cache_write, attn_last_device_error, attn_paged_fwd, attn_prefix_fwd)
from block_sparse_attention_slice_gb300 import binding as B

pytestmark = pytest.mark.gpu
FMTS = ["int8", "e4m3"]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def paged(c, window=0, sinks=0, **kw):
    return attn_paged_fwd(c["q"], c["k"], c["v"], c["d_table"], c["d_lens"], c["scale"], q_ptr=kw.pop("q_ptr", c["d_q_ptr"]),
                          window=window, sinks=sinks, seqs=c["d_seqs"], k_scales=c["ks"], v_scales=c["vs"], **kw)


def prefix(c, **kw):
    return attn_prefix_fwd(c["q"], c["k"], c["v"], c["d_ptable"], c["d_plens"], c["d_first"], c["d_table"], c["d_lens"], c["scale"],
                           q_ptr=kw.pop("q_ptr", c["d_q_ptr"]), seqs=c["d_seqs"], k_scales=c["ks"], v_scales=c["vs"], **kw)


# ---- write, read ------------------------------------------------------------

class Pages:
    """Empty pages in 8 bits; whatever they hold at first, only tokens' places change."""

    def __init__(self, fmt, n_pages, page, hk, d, layout="plain"):
        self.fmt = fmt
        pad, gap = (16, 3) if layout == "heads" else (0, 0)
        self.codes = [torch.full((n_pages, hk, page, d + pad) if pad else (n_pages, page, hk, d), 77, dtype=torch.int8, device="cuda") for _ in range(2)]
        self.s = [torch.full((n_pages, hk, page + gap) if pad else (n_pages, page, hk), -3.0, device="cuda") for _ in range(2)]
        self.k, self.v = (P8.typed(x, fmt)[..., :d].permute(0, 2, 1, 3) if pad else P8.typed(x, fmt) for x in self.codes)
        self.ks, self.vs = (x[..., :page].permute(0, 2, 1) if pad else x for x in self.s)

    def rows(self, x):
        """Codes (bytes) [n_pages, page, hk, d] and scales on the host."""
        i = "kv".index(x)
        return (self.k, self.v)[i].view(torch.int8).cpu().numpy(), (self.ks, self.vs)[i].cpu().numpy()


def tokens(T, hk, d, seed):
    """New rows with what can go wrong among them: nothing but zeros, one value, values far
    apart, halfway between codes, next to the largest and the smallest numbers."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, hk, d)) * np.exp(2 * rng.standard_normal((T, hk, 1)))
    flat = x.reshape(-1, d)
    for i, row in enumerate(flat):
        kind = i % 11
        if kind == 1:
            row[:] = 0
        elif kind == 2:
            row[:] = 0
            row[i % d] = -3.5
        elif kind == 3:      # halfway between codes of int8 and, below, of e4m3
            row[:] = rng.integers(-20, 20, d) + 0.5
            row[i % d] = 127
        elif kind == 4:
            row[:] = rng.integers(8, 120, d) * 2 + 1
            row[i % d] = 448
        elif kind == 5:
            row[:] *= 1e38
        elif kind == 6:
            row[:] *= 1e-38
        elif kind == 7:
            row[:] = 2.0 ** rng.integers(-30, 1, d)
    y = torch.from_numpy(np.clip(x, -3.38e38, 3.38e38).astype(np.float32)).bfloat16()
    return y


WRITE = [([1], [1], 16, 1, 64), ([5, 0, 40], [5, 0, 33], 16, 3, 128), ([70, 129, 16, 17], [1, 1, 1, 1], 64, 8, 128),
         ([300, 7], [280, 0], 32, 5, 64), ([1000], [999], 256, 2, 128), ([33] * 40, [33] * 40, 16, 8, 64)]


@pytest.mark.parametrize("lens,news,page,hk,d", WRITE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("layout", ["plain", "heads"])
def test_write_and_read(lens, news, page, hk, d, fmt, layout):
    c = P.make(lens, news, page, hk, hk, d, seed=3, extra_tokens=2)
    T = c["q"].shape[0]
    k, v = tokens(T, hk, d, 1), tokens(T, hk, d, 2)
    p = Pages(fmt, c["k"].shape[0], page, hk, d, layout)
    was = {x: p.rows(x) for x in "kv"}
    wide = torch.zeros((2, T, hk + 1, d + 8), dtype=torch.bfloat16, device="cuda")      # rows apart in memory
    wide[0, :, :hk, :d], wide[1, :, :hk, :d] = k.cuda(), v.cuda()
    attn_cache_write(p.k, p.v, wide[0, :, :hk, :d], wide[1, :, :hk, :d], c["d_table"], c["d_lens"], q_ptr=c["d_q_ptr"],
                     k_scales=p.ks, v_scales=p.vs)
    assert attn_last_device_error() == 0
    want_rows = {}
    for x, new in (("k", k), ("v", v)):
        codes, scales = (y.copy() for y in was[x])
        enc, sc = oracle.oracle_encode(new.double().numpy(), fmt)
        want_rows[x] = np.full((T, hk, d), np.nan)
        for b, (n, m) in enumerate(zip(lens, news)):
            for t in range(m):
                at = c["table"][b, (n - m + t) // page], (n - m + t) % page
                i = c["q_ptr"][b] + t
                codes[at], scales[at] = enc[i], sc[i]
                want_rows[x][i] = C.values(enc[i], fmt) * sc[i][:, None].astype(np.float64)
        got = p.rows(x)
        # -0 is written for what rounds to zero from below: the same number
        same = C.values(got[0], fmt), C.values(codes, fmt)
        assert np.array_equal(*same, equal_nan=True) and np.array_equal(got[1], scales)
    for dtype in (torch.bfloat16, torch.float32):
        out = [torch.full((T, hk, d), 5.0, dtype=dtype, device="cuda") for _ in range(2)]
        r = attn_cache_read(p.k, p.v, c["d_table"], c["d_lens"], T, q_ptr=c["d_q_ptr"], k_out=out[0], v_out=out[1], k_scales=p.ks, v_scales=p.vs)
        assert r[0] is out[0] and r[1] is out[1] and attn_last_device_error() == 0
        for y, x in zip(out, "kv"):
            w = want_rows[x]
            f32 = torch.from_numpy(np.where(np.isnan(w), 5.0, w).astype(np.float32))
            assert torch.equal(y.cpu(), f32 if dtype == torch.float32 else f32.bfloat16())
    if all(m == 1 for m in news):       # one token each needs no q_ptr
        r = attn_cache_read(p.k, p.v, c["d_table"], c["d_lens"], len(lens), k_scales=p.ks, v_scales=p.vs)
        assert torch.equal(r[0].cpu(), torch.from_numpy(want_rows["k"][2:-2]).float().bfloat16())


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_that_are_not_finite_read_as_nan(fmt):
    p = Pages(fmt, 3, 16, 2, 64)
    k = torch.ones((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    k[0, 1, 5], v[1, 0, 63] = float("inf"), float("nan")
    table, lens, ptr = ints([[2, -1]]), ints([2]), ints([0, 2])
    attn_cache_write(p.k, p.v, k, v, table, lens, q_ptr=ptr, k_scales=p.ks, v_scales=p.vs)
    a, b = attn_cache_read(p.k, p.v, table, lens, 2, q_ptr=ptr, k_scales=p.ks, v_scales=p.vs)
    assert attn_last_device_error() == 0
    assert torch.equal(a.isnan().all(-1).cpu(), torch.tensor([[False, True], [False, False]]))
    assert torch.equal(b.isnan().all(-1).cpu(), torch.tensor([[False, False], [True, False]]))
    assert torch.equal(a[0, 0], k[0, 0]) and not p.rows("k")[0][2, 0, 1].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["plain", "joined", "heads"])
def test_read_pages_of_16_bits(dtype, layout):
    lens, news = [40, 0, 129, 16], [40, 0, 77, 1]
    c = P.make(lens, news, 16, 3, 3, 128, seed=8, slots=[4, 1, 0, 6], layout=layout)
    k, v = attn_cache_read(c["k"], c["v"], c["d_table"], c["d_lens"], sum(news), q_ptr=c["d_q_ptr"], seqs=c["d_seqs"], out_dtype=dtype)
    assert attn_last_device_error() == 0
    for got, x in ((k, "k64"), (v, "v64")):
        want = np.concatenate([oracle.paged.cached_rows(c[x], c["table"][s], n)[n - m:] for s, n, m in zip([4, 1, 0, 6], lens, news)])
        assert got.dtype == dtype and np.array_equal(got.double().cpu().numpy(), want)


def test_bad_places_are_neither_written_nor_read():
    p = Pages("int8", 2, 16, 1, 64)
    x = torch.ones((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    # a page out of range, a slot out of range, more tokens than the length, a good one
    table, lens = ints([[5], [0], [1], [1]]), ints([1, 0, 1, 3])
    out = [torch.full((4, 1, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    seqs = ints([0, 9, 1, 3])
    attn_cache_write(p.k, p.v, x, x, table, lens, seqs=seqs, k_scales=p.ks, v_scales=p.vs)
    assert attn_last_device_error() == B.ATTN_ERR_INVALID_ARG
    codes, scales = p.rows("k")
    assert np.all(codes[1, 2] == 127) and scales[1, 2] == np.float32(1) / np.float32(127)
    codes[1, 2] = 77
    assert np.all(codes == 77) and np.sum(scales != -3) == 1
    attn_cache_read(p.k, p.v, table, lens, 4, seqs=seqs, k_out=out[0], v_out=out[1], k_scales=p.ks, v_scales=p.vs)
    assert attn_last_device_error() == B.ATTN_ERR_INVALID_ARG
    assert torch.all(out[0][:3] == 9) and torch.all(out[0][3] == 1)


# ---- attention --------------------------------------------------------------

ONE = [  # lens, page, hq, hk, d, window, sinks
    ([1], 16, 1, 1, 64, 0, 0), ([17], 16, 4, 1, 128, 0, 0), ([0, 1, 15, 16, 17, 0, 33], 16, 8, 2, 128, 0, 0),
    ([2000], 64, 32, 8, 128, 0, 0), ([2000, 3, 777], 32, 16, 16, 64, 0, 0), ([1030, 60, 5], 16, 6, 2, 64, 64, 4),
    ([1030, 60, 5, 68, 69, 70], 128, 5, 1, 128, 64, 5), ([500, 499], 256, 16, 1, 128, 1, 0), ([500, 499], 16, 20, 1, 64, 1, 1),
    ([513, 40], 16, 4, 2, 128, 37, 100), ([300], 16, 33, 1, 64, 17, 16), ([700], 1024, 8, 8, 128, 2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("lens,page,hq,hk,d,window,sinks", ONE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_token_each(lens, page, hq, hk, d, window, sinks, fmt, dtype):
    c = P8.make(fmt, lens, [1] * len(lens), page, hq, hk, d, seed=len(lens) + d, spread=0.5)
    out, lse = paged(c, window, sinks, q_ptr=None, out_dtype=dtype)
    assert attn_last_device_error() == 0
    P8.check(c, out, lse, P.reference(c, window, sinks))


MANY = [  # lens, news, page, hq, hk, d, window, sinks
    ([40, 3, 9], [5, 3, 9], 16, 4, 2, 64, 0, 0), ([40, 3, 0, 9], [5, 6, 2, 0], 16, 4, 2, 64, 0, 0),
    ([300, 130], [7, 130], 32, 6, 2, 128, 20, 3), ([300, 130], [70, 33], 64, 8, 1, 64, 64, 1),
    ([257], [257], 16, 5, 1, 128, 16, 2), ([600, 200, 50], [200, 1, 50], 128, 16, 4, 128, 100, 7),
    ([1000], [300], 16, 8, 2, 128, 0, 0), ([129, 513], [129, 257], 16, 2, 2, 64, 0, 0), ([400], [65], 256, 40, 1, 64, 50, 0),
    ([3000, 700], [40, 9], 64, 8, 8, 128, 0, 0), ([3000, 700], [40, 9], 32, 4, 2, 64, 0, 0)]


@pytest.mark.parametrize("lens,news,page,hq,hk,d,window,sinks", MANY)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("max_q", [1, None])
def test_several_tokens_each(lens, news, page, hq, hk, d, window, sinks, fmt, max_q):
    c = P8.make(fmt, lens, news, page, hq, hk, d, seed=sum(news) + d, spread=0.5)
    out, lse = paged(c, window, sinks, max_q=max_q)
    assert attn_last_device_error() == 0
    P8.check(c, out, lse, P.reference(c, window, sinks))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("news,max_q", [([1, 1], 1), ([3, 40], 1), ([3, 40], 40), ([200, 150], 200)])
def test_layouts_and_table_rows(fmt, news, max_q):
    c = P8.make(fmt, [900, 333], news, 32, 8, 2, 128, seed=5, layout="heads", slots=[5, 2], extra_tokens=3)
    out = torch.full(c["q"].shape, 7.0, device="cuda")
    lse = torch.full((8, c["q"].shape[0]), 7.0, device="cuda")
    paged(c, 100, 2, out=out, lse=lse, max_q=max_q)
    assert attn_last_device_error() == 0
    assert torch.all(out[:3] == 7) and torch.all(out[-3:] == 7) and torch.all(lse[:, :3] == 7) and torch.all(lse[:, -3:] == 7)
    P8.check(c, out, lse, P.reference(c, 100, 2))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("max_q", [1, 64])
def test_magnitudes_far_apart(fmt, max_q):
    """Rows of keys and values whose scales differ by many powers of ten, large and small queries: the
    weights' own powers of two follow them."""
    c = P8.make(fmt, [700, 90, 1500], [2, 20, 6], 16, 8, 2, 64, seed=12, spread=6.0)
    size = torch.exp(3 * torch.randn(c["q"].shape[:2], generator=torch.Generator().manual_seed(1)))[..., None]
    c["q"] = (c["q"].cpu() * size * 1e-2).bfloat16()
    c["q64"] = c["q"].double().numpy()
    c["q"] = c["q"].cuda()
    out, lse = paged(c, out_dtype=torch.float32, max_q=max_q)
    assert attn_last_device_error() == 0
    P8.check(c, out, lse, P.reference(c))


@pytest.mark.parametrize("fmt", FMTS)
def test_scales_of_zero_and_tiny_and_huge_values(fmt):
    c = P8.make(fmt, [400], [1], 16, 2, 1, 128, seed=2)
    for x, size in (("k", 1e-3), ("v", 1e20)):
        c[x + "s"], c[x + "64"] = c[x + "s"] * size, c[x + "64"] * float(np.float32(size))
    for x in "kv":       # the first hundred tokens are zeros
        for j in range(100):
            at = c["table"][0, j // 16], j % 16
            c[x + "s"][at], c[x + "64"][at] = 0.0, 0.0
    out, lse = paged(c, out_dtype=torch.float32)
    # the scales were multiplied once more: u each
    c["k64"] = c["k64"] * (1 + 2.0 ** -24)
    P8.check(c, out, lse, P.reference(c))
    assert attn_last_device_error() == 0


PRE = [  # plens, first, lens, news, page, hq, hk, d
    ([100], [0, 3], [5, 17, 1], [1, 1, 1], 16, 8, 2, 128), ([700, 33], [0, 2, 5], [40, 3, 9, 60, 1], [3, 1, 2, 5, 1], 16, 4, 4, 64),
    ([2000], [0, 40], [30] * 40, [1] * 40, 64, 8, 1, 128), ([300, 0, 257], [0, 1, 2, 4], [50, 20, 130, 7], [40, 5, 100, 7], 32, 8, 2, 128)]


@pytest.mark.parametrize("plens,first,lens,news,page,hq,hk,d", PRE)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("max_q", [1, None])
def test_prefix(plens, first, lens, news, page, hq, hk, d, fmt, max_q):
    c = P8.make(fmt, lens, news, page, hq, hk, d, seed=4, plens=plens, first=first, spread=0.3)
    out, lse = prefix(c, max_q=max_q)
    assert attn_last_device_error() == 0
    P8.check(c, out, lse, P.reference(c))


@pytest.mark.parametrize("fmt", FMTS)
def test_many_sequences(fmt):
    lens = [1 + i % 40 for i in range(1500)] + [0, 3]
    c = P8.make(fmt, lens, [1] * len(lens), 16, 2, 1, 128, seed=6)
    out, lse = paged(c, q_ptr=None)
    assert attn_last_device_error() == 0
    P8.check(c, out, lse, P.reference(c))


def test_as_many_sequences_as_a_call_takes():
    """The plan of 4096 sequences leaves no room for their records beside the ring."""
    for d in (64, 128):
        lens = [1 + i % 3 for i in range(4096)]
        c = P8.make("int8", lens, [1] * len(lens), 16, 1, 1, d, seed=6)
        out, lse = paged(c, q_ptr=None)
        assert attn_last_device_error() == 0
        P8.check(c, out, lse, P.reference(c))


@pytest.mark.parametrize("max_q", [1, 64])
def test_bad_pages_are_not_followed(max_q):
    c = P8.make("e4m3", [100, 200], [1, 20], 16, 8, 2, 128, seed=7)
    c["d_table"][0, 2] = 1 << 29
    out, lse = paged(c, max_q=max_q)
    assert attn_last_device_error() == B.ATTN_ERR_INVALID_ARG
    ref = P.reference(c)
    rows = slice(int(c["q_ptr"][1]), None)
    whole = (torch.zeros_like(out), torch.zeros_like(lse))
    c1 = dict(c, lens=c["lens"][1:])
    for x, y in zip(whole, (out, lse)):
        x.copy_(y)
    P8.check(c1, out[rows], lse[:, rows], (ref[0][rows], ref[1][:, rows], ref[2][rows], ref[3][:, rows]))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("max_q", [1, 64])
def test_streams_graphs_and_repeats(fmt, max_q):
    c = P8.make(fmt, [900, 333, 40], [20, 7, 1], 16, 8, 2, 128, seed=9)
    want = paged(c, max_q=max_q)
    s = torch.cuda.Stream()
    got = paged(c, max_q=max_q, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):       # two graphs with workspaces of their own
        out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            paged(c, max_q=max_q, out=out, lse=lse)
        graphs.append((g, out, lse))
    for g, out, lse in graphs * 2:
        out.fill_(0), lse.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert attn_last_device_error() == 0


# ---- together ---------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
def test_a_beam_search_over_the_cache(fmt):
    """Prompts written, then steps of: select, reorder pages and states, extend, write, attend.  The
    oracle keeps every beam's own tokens and its rows of keys and values."""
    rng = np.random.default_rng(0)
    G, Bm, hk, hq, d, page, V, n_pages = 3, 4, 2, 8, 64, 16, 50, 80
    rows = G * Bm
    table = torch.full((rows, 8), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    p = Pages(fmt, n_pages, page, hk, d)
    slots = torch.arange(rows, dtype=torch.int32, device="cuda")
    draw = lambda n: torch.from_numpy(rng.standard_normal((n, hk, d)).astype(np.float32)).bfloat16()  # noqa: E731
    enc = lambda x: np.float64(C.values((e := oracle.oracle_encode(x.double().numpy(), fmt))[0], fmt) * e[1][..., None].astype(np.float64))  # noqa: E731

    def write(seqs, counts, k, v):
        attn_cache_extend(table, lens, refs, seqs, ints(counts), page)
        attn_cache_write(p.k, p.v, k.cuda(), v.cuda(), table, lens, q_ptr=ints(np.concatenate([[0], np.cumsum(counts)]).tolist()), seqs=seqs,
                         k_scales=p.ks, v_scales=p.vs)

    kept = []                            # each beam's rows of keys and values
    prompts = [21, 16, 5]
    for g, n in enumerate(prompts):      # every beam of a prompt holds the prompt
        k, v = draw(n), draw(n)
        write(slots[g * Bm:g * Bm + 1], [n], k, v)
        copies = attn_cache_fork(table, lens, refs, slots[g * Bm].repeat(Bm - 1), slots[g * Bm + 1:(g + 1) * Bm], page)
        for pools in ([p.k, p.v], [p.ks, p.vs]):
            attn_cache_copy_pages(pools, copies)
        kept += [(enc(k), enc(v), [])] * Bm
    scores = torch.full((G, Bm), float("-inf"), device="cuda")
    scores[:, 0] = 0
    done = torch.zeros((G, Bm), dtype=torch.bool, device="cuda")
    history = torch.zeros((rows, 6), dtype=torch.int32, device="cuda")
    for step in range(6):
        logits = torch.from_numpy(rng.standard_normal((rows, V)).astype(np.float32) * 2).cuda()
        ref = oracle.oracle_beam_select(logits.double().cpu().numpy(), scores.cpu().numpy(), done.cpu().numpy(), 7)
        scores, parents, toks, done, src = attn_beam_select(logits, scores, done=done, eos=7, slots=slots)
        assert np.array_equal(parents.cpu().numpy(), ref[1]) and np.array_equal(toks.cpu().numpy(), ref[2])
        copies = attn_cache_fork(table, lens, refs, src.view(-1), slots, page)
        for pools in ([p.k, p.v], [p.ks, p.vs]):
            attn_cache_copy_pages(pools, copies)
        attn_beam_reorder([history], parents)
        history[:, step] = toks.view(-1)
        k, v = draw(rows), draw(rows)
        write(slots, [1] * rows, k, v)
        ek, ev = enc(k), enc(v)
        kept = [(np.concatenate([kept[a][0], ek[i:i + 1]]), np.concatenate([kept[a][1], ev[i:i + 1]]), kept[a][2] + [int(t)])
                for i, (a, t) in enumerate(zip(ref[1].ravel(), ref[2].ravel()))]
        q = torch.from_numpy(rng.standard_normal((rows, hq, d)).astype(np.float32)).bfloat16()
        out, lse = attn_paged_fwd(q.cuda(), p.k, p.v, table, lens, 0.125, out_dtype=torch.float32, k_scales=p.ks, v_scales=p.vs)
        assert attn_last_device_error() == 0
        for i, (kk, vv, toks_i) in enumerate(kept):
            assert history[i, :step + 1].tolist() == toks_i and int(lens[i]) == len(kk)
            for h in range(hq):
                x = kk[:, h // (hq // hk)] @ q[i, h].double().numpy() * 0.125
                w = np.exp(x - x.max())
                assert np.abs(out[i, h].double().cpu().numpy() - w @ vv[:, h // (hq // hk)] / w.sum()).max() < 2.0 ** -8 * np.abs(vv).max()
    got = attn_cache_read(p.k, p.v, table, lens, int(lens.sum()), q_ptr=torch.cat([ints([0]), lens.cumsum(0).int()]), out_dtype=torch.float32,
                          k_scales=p.ks, v_scales=p.vs)
    for y, i in zip(got, (0, 1)):
        assert np.array_equal(y.cpu().numpy(), np.concatenate([x[i] for x in kept]).astype(np.float32))
