"""The cache in 8 bits where it can go wrong: waits that run out, layouts with strides of
zero, table rows of many pages for short sequences, bad places, several calls at once,
captured ones, offsets past 32 bits, and what the Python entry points refuse."""
import numpy as np
import pytest
import torch

import oracle
import paged8_cases as P8
import paged_cases as P
from block_sparse_attention_slice_gb300 import AttnError, attn_cache_read, attn_cache_write, attn_last_device_error, attn_set_wait_limit_ns
from block_sparse_attention_slice_gb300 import binding as B
from test_gpu_cache8 import FMTS, Pages, ints, paged, prefix, tokens

pytestmark = pytest.mark.gpu
WIDE = 400000      # keys that a table row of this width could hold: a call that is not a short one


def widen(c, keys=WIDE):
    """The table with more columns, which no length reaches: long sequences are possible then, and the
    kernel for them is taken."""
    for name in ("d_table", "d_ptable"):
        t = c[name]
        c[name] = torch.cat([t, torch.full((t.shape[0], -(-keys // c["k"].shape[1])), 1 << 28, dtype=torch.int32, device="cuda")], 1).contiguous()
    return c


@pytest.mark.parametrize("lens,page,hq,hk,d,window,sinks", [
    ([1], 16, 1, 1, 64, 0, 0), ([1], 16, 8, 1, 128, 0, 0), ([0, 2, 31, 32, 33], 16, 4, 1, 64, 0, 0), ([15, 16, 17, 0, 64, 65], 64, 8, 2, 128, 0, 0),
    ([500, 3, 129], 32, 21, 3, 64, 0, 0), ([777, 1200], 256, 16, 8, 128, 0, 0), ([3000], 16, 7, 7, 128, 0, 0), ([4096, 4095, 31], 128, 32, 8, 64, 0, 0)])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_short_sequences_of_wide_tables(lens, page, hq, hk, d, window, sinks, fmt, dtype):
    c = widen(P8.make(fmt, lens, [1] * len(lens), page, hq, hk, d, seed=sum(lens) + d, spread=0.5))
    out, lse = paged(c, window, sinks, q_ptr=None, out_dtype=dtype)
    assert attn_last_device_error() == 0
    P8.check(c, out, lse, P.reference(c, window, sinks))


@pytest.mark.parametrize("page,d,fmt", [(16, 64, "int8"), (32, 128, "e4m3")])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 0), (33, 3), (20, 40), (64, 1)])
def test_windows_of_many_sequences(page, d, window, sinks, fmt):
    lens = [(37 * i) % 150 for i in range(900)]
    c = widen(P8.make(fmt, lens, [1] * len(lens), page, 16, 8, d, seed=window + d, spread=0.5))
    out, lse = paged(c, window, sinks, q_ptr=None)
    assert attn_last_device_error() == 0
    P8.check(c, out, lse, P.reference(c, window, sinks))


@pytest.mark.parametrize("lens,news,page,hq,hk,d,window,sinks", [
    ([40, 3, 9], [5, 3, 9], 16, 4, 2, 64, 0, 0), ([300, 130, 0, 5], [7, 8, 1, 6], 32, 8, 2, 64, 20, 3), ([257, 1000], [4, 4], 64, 20, 4, 64, 0, 0),
    ([3000, 33], [2, 2], 16, 16, 2, 64, 700, 1), ([900, 70], [3, 4], 128, 40, 8, 128, 0, 0), ([5000], [16], 256, 4, 2, 64, 0, 0), ([40] * 70, [5] * 70, 16, 8, 2, 64, 9, 1)])
@pytest.mark.parametrize("fmt", FMTS)
def test_up_to_32_rows_of_wide_tables(lens, news, page, hq, hk, d, window, sinks, fmt):
    c = widen(P8.make(fmt, lens, news, page, hq, hk, d, seed=sum(news) + d, spread=0.5))
    out, lse = paged(c, window, sinks, max_q=min(max(news), 32 * hk // hq))
    assert attn_last_device_error() == 0
    P8.check(c, out, lse, P.reference(c, window, sinks))


@pytest.mark.parametrize("keys", [3000, 12000, 30000])
@pytest.mark.parametrize("news", [[1, 1, 1], [4, 3, 1], [7, 2, 5]])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", FMTS)
def test_tables_between_narrow_and_wide(keys, news, d, fmt):
    c = widen(P8.make(fmt, [2700, 333, 16], news, 16, 8, 2, d, seed=keys + d, spread=0.5), keys)
    for window, sinks in ((0, 0), (2500, 3)):
        out, lse = paged(c, window, sinks, max_q=max(news))
        assert attn_last_device_error() == 0
        P8.check(c, out, lse, P.reference(c, window, sinks))


@pytest.mark.parametrize("news", [[2, 2, 1], [1, 0, 2], [7, 5, 1]])
@pytest.mark.parametrize("fmt", FMTS)
def test_a_few_tokens_of_few_heads(news, fmt):
    """Rows of several tokens in one tile of 8, with masks of their own; tokens before the first key."""
    c = widen(P8.make(fmt, [700, 4, 2], news, 16, 6, 2, 128, seed=4, spread=0.5, extra_tokens=2))
    for window, sinks in ((0, 0), (9, 2)):
        for max_q in (1, 2, 7):
            out, lse = paged(c, window, sinks, max_q=max_q)
            assert attn_last_device_error() == 0
            P8.check(c, out, lse, P.reference(c, window, sinks))


@pytest.mark.parametrize("news", [[1, 1], [1, 6], [6, 3], [30, 50], [100, 4]])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", FMTS)
def test_strides_of_zero(news, d, fmt):
    """All heads see one head's pages, or every page of the table the same memory."""
    for what in ("head", "page"):
        c = P8.make(fmt, [2000, 900] if what == "head" else [16, 16], news if what == "head" else [1, 6 if max(news) > 1 else 1], 16, 16,
                    1 if what == "head" else 4, d, seed=3, spread=0.3)
        ref_pages = {}
        if what == "head":
            for x in "kv":
                c[x], c[x + "s"] = c[x].expand(-1, -1, 4, -1), c[x + "s"].expand(-1, -1, 4)
                c[x + "64"] = np.broadcast_to(c[x + "64"], c[x + "64"].shape[:2] + (4, d))
        else:
            at = int(c["table"][0, 0])
            for x in "kv":
                ref_pages[x] = c[x + "64"][at]
                c[x], c[x + "s"] = c[x][at:at + 1].expand(9, -1, -1, -1), c[x + "s"][at:at + 1].expand(9, -1, -1)
                c[x + "64"] = np.broadcast_to(ref_pages[x], (9,) + ref_pages[x].shape)
            c["table"] = (np.arange(2 * 150) % 9).reshape(2, 150).astype(np.int32)
            c["lens"] = np.asarray([2000, 900], np.int32)
            c["d_table"], c["d_lens"] = torch.from_numpy(c["table"]).cuda(), torch.from_numpy(c["lens"]).cuda()
        out, lse = paged(widen(c))
        assert attn_last_device_error() == 0
        P8.check(c, out, lse, P.reference(c))
        k, v = attn_cache_read(c["k"], c["v"], c["d_table"], c["d_lens"], len(c["q"]), q_ptr=c["d_q_ptr"], out_dtype=torch.float32,
                               k_scales=c["ks"], v_scales=c["vs"])
        assert attn_last_device_error() == 0
        for y, x in ((k, "k64"), (v, "v64")):       # code * scale rounded once, to f32
            for b, n in enumerate(c["lens"]):
                rows = oracle.paged.cached_rows(c[x], c["table"][b], n)[n - (c["q_ptr"][b + 1] - c["q_ptr"][b]):]
                assert np.array_equal(y[c["q_ptr"][b]:c["q_ptr"][b + 1]].cpu().numpy(), rows.astype(np.float32))


# ---- waits ------------------------------------------------------------------

def cases_of_waits(fmt, news):
    """A paged and a prefix call, each with the kernel that `news` tokens go to."""
    c = P8.make(fmt, [12000, 9000], [news, news], 64, 16, 2, 128, seed=7)
    pre = P8.make(fmt, [news, news], [news, news], 64, 16, 2, 128, seed=7, plens=[12000, 12000] if news == 1 else [4000],
                  first=[0, 1, 2] if news == 1 else [0, 2])
    return widen(c), widen(pre)


@pytest.mark.parametrize("news", [1, 6, 100])       # a few rows, one row tile an item, two
@pytest.mark.parametrize("fmt", FMTS)
def test_a_load_that_never_comes_ends_in_a_timeout(news, fmt, monkeypatch):
    # ATTN_TEST_STALL_PAGED leaves a load out: the bounded wait for it runs out, the launch ends
    # with all others landed and the status says so; the next call is as before
    c, pre = cases_of_waits(fmt, news)
    a, b = paged(c, max_q=news), prefix(pre, max_q=news)
    assert attn_last_device_error() == 0
    attn_set_wait_limit_ns(50_000_000)
    monkeypatch.setenv("ATTN_TEST_STALL_PAGED", "1")
    try:
        for call in (lambda: paged(c, max_q=news), lambda: prefix(pre, max_q=news)):
            call()
            assert attn_last_device_error() == B.ATTN_ERR_TIMEOUT
    finally:
        monkeypatch.delenv("ATTN_TEST_STALL_PAGED")
        attn_set_wait_limit_ns(4_000_000_000)
    for x, y in zip(a + b, paged(c, max_q=news) + prefix(pre, max_q=news)):
        assert torch.equal(x, y)
    assert attn_last_device_error() == 0


@pytest.mark.parametrize("news", [1, 6, 100])
@pytest.mark.parametrize("fmt", FMTS)
def test_the_shortest_wait_limit_ends_a_call_in_its_result_or_in_a_timeout(news, fmt):
    c, pre = cases_of_waits(fmt, news)
    want = paged(c, max_q=news) + prefix(pre, max_q=news)
    assert attn_last_device_error() == 0
    for _ in range(10):
        attn_set_wait_limit_ns(1000)         # the least that is taken
        try:
            got = paged(c, max_q=news) + prefix(pre, max_q=news)
            status = attn_last_device_error()
        finally:
            attn_set_wait_limit_ns(4_000_000_000)
        assert status in (0, B.ATTN_ERR_TIMEOUT)
        if status == 0:
            assert all(torch.equal(x, y) for x, y in zip(want, got))
        assert all(torch.equal(x, y) for x, y in zip(want, paged(c, max_q=news) + prefix(pre, max_q=news)))
        assert attn_last_device_error() == 0


# ---- bad places, rows that see nothing -----------------------------------------

@pytest.mark.parametrize("what", ["slot", "length", "negative length", "page", "negative page", "q_ptr", "q_ptr end"])
@pytest.mark.parametrize("max_q,wide", [(1, False), (1, True), (5, False), (20, False)])
def test_bad_device_contents_are_reported_and_read_nothing(what, max_q, wide):
    c = P8.make("e4m3", [70, 33, 90], [2, 20, 1], 16, 8, 2, 128, seed=8, slots=[0, 1, 2])
    ref = P.reference(c)
    if wide:
        widen(c)
    if what == "slot":
        c["d_seqs"][1] = 99
    elif what == "length":
        c["d_lens"][1] = 16 * c["d_table"].shape[1] + 1
    elif what == "negative length":
        c["d_lens"][1] = -5
    elif what == "page":
        c["d_table"][1, 1] = c["k"].shape[0]
    elif what == "negative page":
        c["d_table"][1, 1] = -1
    elif what == "q_ptr":
        c["d_q_ptr"][1] = -1
    elif what == "q_ptr end":
        c["d_q_ptr"][3] = 10 ** 6
    out, lse = paged(c, max_q=max_q)
    assert attn_last_device_error() == B.ATTN_ERR_INVALID_ARG
    assert attn_last_device_error() == 0
    fine = {"q_ptr": [2], "q_ptr end": [0, 1]}.get(what, [0, 2])       # sequences that are served
    for b in range(3):
        if b not in fine:
            for x in ref:
                (x if x.shape[0] == len(c["q"]) else x.T)[c["q_ptr"][b]:c["q_ptr"][b + 1]] = np.nan
    P8.check(c, out, lse, ref)
    if what in ("slot", "length", "negative length"):
        rows = slice(c["q_ptr"][1], c["q_ptr"][2])
        assert torch.all(out[rows] == 0) and torch.all(torch.isneginf(lse[:, rows]))


@pytest.mark.parametrize("lens,news,hq,hk,d,max_q", [
    ([3, 40], [6, 2], 4, 2, 64, 1), ([3, 0], [6, 2], 8, 1, 128, 2), ([3, 0], [6, 2], 8, 1, 128, 6), ([20, 9], [50, 12], 8, 2, 128, 50),
    ([20, 9], [90, 100], 8, 2, 64, 100)])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("wide", [False, True])
def test_a_token_that_sees_nothing_gets_zeros(lens, news, hq, hk, d, max_q, fmt, wide):
    c = P8.make(fmt, lens, news, 16, hq, hk, d, seed=3)
    out, lse = paged(widen(c) if wide else c, max_q=max_q)
    assert attn_last_device_error() == 0
    P8.check(c, out, lse, P.reference(c))
    none = torch.from_numpy(np.concatenate([np.arange(new) < new - n for n, new in zip(lens, news)])).cuda()
    assert torch.all(out[none] == 0) and torch.all(torch.isneginf(lse[:, none]))


# ---- streams, graphs, sizes ---------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
def test_calls_at_once_with_their_own_workspaces(fmt):
    c = widen(P8.make(fmt, [30000, 40, 900], [1, 1, 1], 16, 8, 2, 128, seed=9))
    pre = P8.make(fmt, [1000, 40, 900, 5] * 6, [1] * 24, 16, 32, 8, 128, seed=9, plens=[5000, 700], first=[0, 16, 24])
    ref = P.reference(c), P.reference(pre)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [(paged(c, q_ptr=None, stream=streams[i % 3]), prefix(pre, stream=streams[(i + 1) % 3])) for i in range(9)]
    torch.cuda.synchronize()
    P8.check(c, *got[0][0], ref[0])
    P8.check(pre, *got[0][1], ref[1])
    for a in got[1:]:
        for x, y in zip(a[0] + a[1], got[0][0] + got[0][1]):
            assert torch.equal(x, y)
    assert attn_last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hq,new", [(4, 1), (16, 6)])
def test_written_attended_to_and_read_in_one_graph(fmt, hq, new):
    """A step as a server captures it; what the lists and the rows hold when it is replayed counts."""
    lens, hk, d, page = [900, 333, 40], 2, 128, 16
    c = widen(P8.make(fmt, lens, [new] * 3, page, hq, hk, d, seed=5))
    x = [tokens(3 * new, hk, d, s).cuda() for s in (1, 2)]
    both = dict(k_scales=c["ks"], v_scales=c["vs"])

    def step(stream=None):
        attn_cache_write(c["k"], c["v"], *x, c["d_table"], c["d_lens"], q_ptr=c["d_q_ptr"], stream=stream, **both)
        return paged(c, max_q=new, stream=stream) + attn_cache_read(c["k"], c["v"], c["d_table"], c["d_lens"], 3 * new, q_ptr=c["d_q_ptr"],
                                                                  stream=stream, **both)

    g = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        held = step()
    for seed in range(3):
        gen = torch.Generator().manual_seed(seed)
        for y in x:
            y.copy_(torch.randn(y.shape, generator=gen))
        c["d_lens"] -= 1          # one token earlier each time
        g.replay()
        torch.cuda.synchronize()
        got = [y.clone() for y in held]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        want = step(s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for y, z in zip(got[2:], x):       # half a step of 254, or of e4m3 (2^-4 of the value, or half its least step), and bf16's
            top = z.float().abs().amax(-1, keepdim=True)
            step8 = top / 254 if fmt == "int8" else torch.maximum(z.float().abs() / 16, top / 448 * 2.0 ** -10)
            assert torch.all((y.float() - z.float()).abs() <= step8 * (1 + 2.0 ** -7) + z.float().abs() * 2.0 ** -7)
    assert attn_last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(fmt):
    """Pages that begin beyond 2^32 bytes: the same bits as of pages that lie near."""
    page, hk, d, n_pages = 256, 8, 128, 17000
    big = [P8.typed(torch.empty((n_pages, page, hk, d), dtype=torch.int8, device="cuda"), fmt) for _ in range(2)]
    scales = [torch.empty((n_pages, page, hk), device="cuda") for _ in range(2)]
    assert (n_pages - 3) * page * hk * d > 2 ** 32
    small = Pages(fmt, 3, page, hk, d)
    far, near = ints([[n_pages - 1, 0, n_pages - 2]]), ints([[0, 1, 2]])
    lens = ints([700])
    gen = torch.Generator().manual_seed(0)
    new = [torch.randn((700, hk, d), generator=gen).bfloat16().cuda() for _ in range(2)]
    ptr = ints([0, 700])
    attn_cache_write(*big, *new, far, lens, q_ptr=ptr, k_scales=scales[0], v_scales=scales[1])
    attn_cache_write(small.k, small.v, *new, near, lens, q_ptr=ptr, k_scales=small.ks, v_scales=small.vs)
    a = attn_cache_read(*big, far, lens, 700, q_ptr=ptr, k_scales=scales[0], v_scales=scales[1])
    b = attn_cache_read(small.k, small.v, near, lens, 700, q_ptr=ptr, k_scales=small.ks, v_scales=small.vs)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    wide = torch.cat([far, torch.full((1, 200), -1, dtype=torch.int32, device="cuda")], 1)
    wide = torch.cat([wide] + [wide[:, -1:].expand(-1, 1200)], 1).contiguous()
    for n, hq in ((1, 32), (4, 32), (40, 32)):
        q = torch.randn((n, hq, d), generator=gen).bfloat16().cuda()
        for t in (far, wide):
            c = dict(q=q, k=big[0], v=big[1], ks=scales[0], vs=scales[1], d_table=t, d_lens=lens, scale=0.1, d_seqs=None, d_q_ptr=ints([0, n]))
            x = paged(c)
            c.update(k=small.k, v=small.v, ks=small.ks, vs=small.vs, d_table=torch.where(t == n_pages - 1, 0, torch.where(t == 0, 1, torch.where(t == n_pages - 2, 2, t))))
            y = paged(c)
            assert all(torch.equal(u, w) for u, w in zip(x, y))
    assert attn_last_device_error() == 0


def test_more_heads_than_a_cache_call_takes_are_refused():
    s = torch.zeros((1, 16, 1025), device="cuda")
    k = torch.zeros((1, 16, 1025, 64), dtype=torch.int8, device="cuda")
    x = torch.zeros((1, 1025, 64), dtype=torch.bfloat16, device="cuda")
    one = ints([[0]]), ints([1])
    for call in (lambda: attn_cache_write(k, k, x, x, *one, k_scales=s, v_scales=s), lambda: attn_cache_read(k, k, *one, 1, k_scales=s, v_scales=s)):
        with pytest.raises(AttnError) as e:
            call()
        assert e.value.code == B.ATTN_ERR_UNSUPPORTED


@pytest.mark.parametrize("fmt", FMTS)
def test_as_many_heads_as_a_cache_call_takes(fmt):
    """A token of 1024 heads is read back; of the numbers of words a token and a head each reciprocal is right."""
    for hk, d in ((1024, 64), (1024, 128), (1023, 128), (7, 64), (1, 64)):
        p = Pages(fmt, 40, 16, hk, d)
        n = 600 if hk < 1000 else 30
        x = [torch.randn((n, hk, d), generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(2)]
        table, lens, ptr = torch.arange(40, dtype=torch.int32, device="cuda")[None], ints([n]), ints([0, n])
        attn_cache_write(p.k, p.v, *x, table, lens, q_ptr=ptr, k_scales=p.ks, v_scales=p.vs)
        got = attn_cache_read(p.k, p.v, table, lens, n, q_ptr=ptr, k_scales=p.ks, v_scales=p.vs, out_dtype=torch.float32)
        for name, y, z in zip("kv", got, x):
            codes, scales = oracle.oracle_encode(z.double().cpu().numpy(), fmt)
            c, s = p.rows(name)
            assert np.array_equal(c.reshape(-1, hk, d)[:n], codes) and np.array_equal(s.reshape(-1, hk)[:n], scales)
            assert torch.equal(y, (P8.typed(torch.from_numpy(codes), fmt).float() * torch.from_numpy(scales)[..., None]).cuda())
    assert attn_last_device_error() == 0


# ---- refusals of the Python entry points ---------------------------------------

def test_refusals():
    c = P8.make("int8", [40, 9], [1, 1], 16, 4, 2, 64, seed=1)
    paged(c, q_ptr=None)
    k, ks = c["k"], c["ks"]
    for bad in (dict(ks=None), dict(vs=None), dict(ks=None, vs=None), dict(ks=ks.double()), dict(ks=ks.cpu()), dict(ks=ks[:, :, :1]), dict(vs=ks[:-1]),
                dict(ks=ks.transpose(0, 1).contiguous().transpose(0, 1)), dict(k=k.view(torch.uint8)), dict(k=k.view(torch.float8_e4m3fn)),
                dict(k=k.bfloat16(), v=k.bfloat16()), dict(k=k.view(torch.float8_e5m2), v=k.view(torch.float8_e5m2))):
        with pytest.raises(ValueError):
            paged({**c, **bad}, q_ptr=None)
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    both = dict(k_scales=ks, v_scales=ks)
    for bad in (x.float(), x[:1, :1], x.cpu(), x[..., :32]):
        with pytest.raises(ValueError):
            attn_cache_write(k, c["v"], bad, bad, c["d_table"], c["d_lens"], **both)
    read = lambda **kw: attn_cache_read(**{**dict(k_pages=k, v_pages=c["v"], table=c["d_table"], seq_lens=c["d_lens"], n_tokens=2), **both, **kw})  # noqa: E731
    read()
    for bad in (dict(n_tokens=-1), dict(out_dtype=torch.float16), dict(k_out=x), dict(k_out=x, v_out=x.float()), dict(k_out=x[:1], v_out=x[:1]),
                dict(k_out=x, v_out=x, out_dtype=torch.float32), dict(k_out=x.cpu(), v_out=x.cpu()), dict(q_ptr=ints([0, 2])), dict(q_ptr=ints([0, 1, 2]).long()),
                dict(seqs=ints([[0, 1]]))):
        with pytest.raises(ValueError):
            read(**bad)
    for bad in (dict(n_tokens=3), dict(n_tokens=1)):       # no q_ptr: one token a sequence
        with pytest.raises(AttnError):
            read(**bad)
    with pytest.raises(TypeError):
        read(n_tokens=2.5)
    assert attn_last_device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("max_q,wide", [(1, False), (1, True), (4, False), (20, False)])
@pytest.mark.parametrize("size", [2.0 ** 118, 2.0 ** -133])
def test_queries_as_large_and_as_small_as_they_come(fmt, max_q, wide, size):
    """Large: scores of 1e11 and more, of which the largest alone has a weight; it is rounded once, to bf16 at
    the coarsest (2^-8).  Small: all scores are 0 to within 1e-30, every weight is 1."""
    c = P8.make(fmt, [500, 77], [1, 1], 16, 4, 1, 64, seed=3)
    down = torch.tensor(1e-24 if size > 1 else 1.0)
    c["ks"], c["k64"] = c["ks"] * down.cuda(), c["k64"] * down.double().item()
    c["q"] = (c["q"].cpu().double() * size).bfloat16()
    c["q64"] = c["q"].double().numpy()
    c["q"] = c["q"].cuda()
    assert np.isfinite(c["q64"]).all() and np.any(c["q64"])
    out, lse = paged(widen(c) if wide else c, out_dtype=torch.float32, max_q=max_q)
    assert attn_last_device_error() == 0
    O, L, A, _ = P.reference(c)
    if size > 1:
        for b, n in enumerate(c["lens"]):       # the inputs leave one key a weight
            k = oracle.paged.cached_rows(c["k64"], c["table"][b], n)[:, 0]
            s = np.sort(k @ c["q64"][b].T * c["scale"], axis=0)
            assert np.all(s[-1] - s[-2] > 1e7) and np.all(s[-1] - s[-2] > 2.0 ** -12 * np.abs(s[-1]))
    # weights, and sums of up to 500 f32 terms
    assert np.all(np.abs(out.double().cpu().numpy() - O) <= (2.0 ** -8 + 500 * 2.0 ** -24) * A)
    assert np.all(np.abs(lse.double().cpu().numpy() - L) <= 2.0 ** -16 * np.abs(L) + 2.0 ** -20)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("times", [1, 4])       # a call of few tokens, one that fills the GPU
def test_every_pair_of_significands(fmt, times):
    """A row's largest value and each of its others in all 128 x 128 significands that bf16 has, the others up to 2^12 times
    smaller: every quotient that lies halfway between two codes is among them."""
    sig = 1 + np.arange(128) / 128
    rows = []
    for a in sig:
        for e in range(13):
            x = sig * 2.0 ** -e * np.where(np.arange(128) % 2, -1, 1)
            top = np.where(np.abs(x) <= a, x, x / 2)
            for at in (0, 127):
                y = top.copy()
                y[at] = a
                rows.append(y)
    x = torch.from_numpy(np.stack(rows).reshape(-1, 2, 128)).bfloat16().repeat(times, 1, 1)
    n = len(x)
    k, v = x.cuda(), (x.float() * 2.0 ** 90).bfloat16().cuda()
    p = Pages(fmt, -(-n // 64), 64, 2, 128)
    table, lens, ptr = torch.arange(-(-n // 64), dtype=torch.int32, device="cuda")[None], ints([n]), ints([0, n])
    attn_cache_write(p.k, p.v, k, v, table, lens, q_ptr=ptr, k_scales=p.ks, v_scales=p.vs)
    assert attn_last_device_error() == 0
    for name, z in (("k", k), ("v", v)):
        codes, scales = oracle.oracle_encode(z.double().cpu().numpy(), fmt)
        c, s = p.rows(name)
        assert np.array_equal(c.reshape(-1, 2, 128)[:n], codes) and np.array_equal(s.reshape(-1, 2)[:n], scales)
