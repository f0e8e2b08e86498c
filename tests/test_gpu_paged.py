"""Attention over a paged cache against the float64 oracle: window, first
tokens, ragged batches, shared prefixes, layouts, and what a cache holds in
places that no token owns."""
import numpy as np
import pytest
import torch

import oracle
import paged_cases as P
from block_sparse_attention_slice_gb300 import (attn_build_tiles, attn_bwd, attn_fwd, attn_last_device_error, attn_paged_fwd,
                                                attn_prefix_fwd, attn_set_wait_limit_ns, attn_slices_from_windows)
from block_sparse_attention_slice_gb300 import binding as B

pytestmark = pytest.mark.gpu


def paged(c, window=0, sinks=0, **kw):
    return attn_paged_fwd(c["q"], c["k"], c["v"], c["d_table"], c["d_lens"], c["scale"], q_ptr=kw.pop("q_ptr", c["d_q_ptr"]),
                          window=window, sinks=sinks, seqs=c["d_seqs"], **kw)


def prefix(c, **kw):
    return attn_prefix_fwd(c["q"], c["k"], c["v"], c["d_ptable"], c["d_plens"], c["d_first"], c["d_table"], c["d_lens"],
                           c["scale"], q_ptr=kw.pop("q_ptr", c["d_q_ptr"]), seqs=c["d_seqs"], **kw)


ONE = [  # lens, page, hq, hk, d, window, sinks
    ([1], 16, 1, 1, 64, 0, 0), ([17], 16, 4, 1, 128, 0, 0), ([0, 1, 15, 16, 17, 0, 33], 16, 8, 2, 128, 0, 0),
    ([2000], 64, 32, 8, 128, 0, 0), ([2000, 3, 777], 32, 16, 16, 64, 0, 0), ([1030, 60, 5], 16, 6, 2, 64, 64, 4),
    ([1030, 60, 5, 68, 69, 70], 128, 5, 1, 128, 64, 5), ([500, 499], 256, 16, 1, 128, 1, 0), ([500, 499], 16, 20, 1, 64, 1, 1),
    ([513, 40], 16, 4, 2, 128, 37, 100), ([300], 16, 33, 1, 64, 17, 16), ([700], 1024, 8, 8, 128, 2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("lens,page,hq,hk,d,window,sinks", ONE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_token_each(lens, page, hq, hk, d, window, sinks, dtype):
    c = P.make(lens, [1] * len(lens), page, hq, hk, d, seed=len(lens) + d)
    out, lse = paged(c, window, sinks, q_ptr=None, out_dtype=dtype)
    assert attn_last_device_error() == 0
    P.check(c, out, lse, P.reference(c, window, sinks))


MANY = [  # lens, news, page, hq, hk, d, window, sinks
    ([40, 3, 9], [5, 3, 9], 16, 4, 2, 64, 0, 0), ([40, 3, 0, 9], [5, 6, 2, 0], 16, 4, 2, 64, 0, 0),
    ([300, 130], [7, 130], 32, 6, 2, 128, 20, 3), ([300, 130], [70, 33], 64, 8, 1, 64, 64, 1),
    ([257], [257], 16, 5, 1, 128, 16, 2), ([600, 200, 50], [200, 1, 50], 128, 16, 4, 128, 100, 7),
    ([1000], [300], 16, 8, 2, 128, 0, 0), ([129, 513], [129, 257], 16, 2, 2, 64, 0, 0), ([400], [65], 256, 40, 1, 64, 50, 0)]


@pytest.mark.parametrize("lens,news,page,hq,hk,d,window,sinks", MANY)
@pytest.mark.parametrize("max_q", [1, None])
def test_several_tokens_each(lens, news, page, hq, hk, d, window, sinks, max_q):
    c = P.make(lens, news, page, hq, hk, d, seed=sum(news) + d)
    out, lse = paged(c, window, sinks, max_q=max_q)
    assert attn_last_device_error() == 0
    P.check(c, out, lse, P.reference(c, window, sinks))


@pytest.mark.parametrize("layout", ["plain", "joined", "heads"])
@pytest.mark.parametrize("garbage", [float("nan"), float("inf"), 0.0])
@pytest.mark.parametrize("max_q", [1, 40])
def test_layouts_slots_and_rows_of_no_sequence(layout, garbage, max_q):
    lens, news = [70, 9, 200], [3, 9, 40]
    c = P.make(lens, news, 32, 8, 2, 128, seed=5, slots=[4, 0, 7], layout=layout, garbage=garbage, extra_tokens=3)
    T = c["q"].shape[0]
    out = torch.full((T, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, T), 7.0, device="cuda")
    paged(c, 33, 2, out=out, lse=lse, max_q=max_q)
    assert attn_last_device_error() == 0
    P.check(c, out, lse, P.reference(c, 33, 2))
    for x in (out[:3], out[-3:], lse[:, :3], lse[:, -3:]):
        assert torch.all(x == 7.0)


@pytest.mark.parametrize("n", [1, 300, 1500, 4096])
def test_many_sequences(n):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 40, n).tolist()
    c = P.make(lens, [1] * n, 16, 2, 1, 64, seed=n)
    out, lse = paged(c, 19, 2, q_ptr=None)
    assert attn_last_device_error() == 0
    P.check(c, out, lse, P.reference(c, 19, 2))


@pytest.mark.parametrize("n,d", [(40, 64), (1500, 128), (2500, 64), (4096, 64), (4096, 128)])
@pytest.mark.parametrize("max_q", [3, 40])       # one row tile an item, two
def test_many_sequences_of_several_tokens(n, d, max_q):
    rng = np.random.default_rng(n)
    news = rng.integers(0, 4, n).tolist()
    c = P.make(rng.integers(0, 60, n).tolist(), news, 16, 8, 1, d, seed=n)
    out, lse = paged(c, 19, 2, max_q=max_q)
    assert attn_last_device_error() == 0
    P.check(c, out, lse, P.reference(c, 19, 2))


@pytest.mark.parametrize("n,groups", [(600, 130), (4096, 1500)])
def test_many_groups_of_several_tokens(n, groups):
    # the prefixes on the tensor cores, and what follows them on either kernel
    rng = np.random.default_rng(n)
    first = np.sort(rng.integers(0, n + 1, groups + 1)).tolist()
    c = P.make(rng.integers(0, 40, n).tolist(), rng.integers(0, 4, n).tolist(), 16, 8, 1, 64, seed=n,
               plens=rng.integers(0, 60, groups).tolist(), first=first)
    ref = P.reference(c)
    for max_q in (1, 3):
        out, lse = prefix(c, max_q=max_q)
        assert attn_last_device_error() == 0
        P.check(c, out, lse, ref)


@pytest.mark.parametrize("hq,hk,d,page,news", [(8, 2, 128, 64, 1), (3, 1, 64, 16, 1), (16, 4, 128, 16, 37), (32, 8, 64, 512, 130)])
def test_long_sequence_alone(hq, hk, d, page, news):
    # one sequence: every span of every worker is a piece of its few items
    c = P.make([20011], [news], page, hq, hk, d, seed=3)
    ref = P.reference(c)
    for dtype in (torch.bfloat16, torch.float32):
        out, lse = paged(c, out_dtype=dtype)
        P.check(c, out, lse, ref)
    again = paged(c, out_dtype=torch.float32)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)       # the same bits every time
    assert attn_last_device_error() == 0


PRE = [  # plens, first, lens, news, page, hq, hk, d
    ([100], [0, 3], [5, 1, 33], [1, 1, 1], 16, 4, 1, 64), ([1000], [0, 16], list(range(1, 17)), [1] * 16, 32, 32, 8, 128),
    ([0, 50, 129], [0, 1, 1, 4], [7, 8, 9, 40], [1, 2, 3, 4], 16, 8, 2, 128),
    ([300, 17], [1, 3, 4], [5, 6, 0, 2, 90], [1, 2, 2, 1, 3], 16, 6, 2, 64),     # the first and last in no group
    ([700], [0, 40], [20] * 40, [5] * 40, 64, 8, 1, 128), ([64, 64], [0, 1, 2], [3, 4], [3, 4], 64, 40, 1, 64),
    ([2500], [0, 2], [600, 300], [300, 300], 128, 4, 2, 128)]


@pytest.mark.parametrize("plens,first,lens,news,page,hq,hk,d", PRE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_shared_prefix(plens, first, lens, news, page, hq, hk, d, dtype):
    c = P.make(lens, news, page, hq, hk, d, seed=len(lens), plens=plens, first=first)
    out, lse = prefix(c, out_dtype=dtype)
    assert attn_last_device_error() == 0
    P.check(c, out, lse, P.reference(c))


@pytest.mark.parametrize("plens,first,lens,news,hq,hk,d", [
    ([20000], [0, 20], [1] * 20, [1] * 20, 32, 8, 128), ([20000], [0, 20], [0] * 20, [1] * 20, 32, 8, 128),
    ([1], [0, 6], [9000] * 6, [1] * 6, 32, 8, 128), ([0], [0, 6], [9000] * 6, [1] * 6, 32, 8, 128),
    ([0, 0], [0, 9, 20], [0] * 20, [1] * 20, 16, 4, 64), ([9000, 0, 3], [0, 7, 30, 40], [7000] + [1] * 39, [2] * 40, 8, 8, 64)])
def test_prefixes_and_what_follows_of_any_proportion(plens, first, lens, news, hq, hk, d):
    # the two passes of the call share the GPU by how many keys each has
    c = P.make(lens, news, 16, hq, hk, d, seed=4, plens=plens, first=first)
    out, lse = prefix(c)
    assert attn_last_device_error() == 0
    P.check(c, out, lse, P.reference(c))
    again = prefix(c)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_no_prefix_at_all_equals_the_paged_call():
    c = P.make([50, 60], [1, 1], 16, 8, 2, 128, seed=1)
    none = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    a = attn_prefix_fwd(c["q"], c["k"], c["v"], none, torch.empty(0, dtype=torch.int32, device="cuda"),
                        torch.zeros(1, dtype=torch.int32, device="cuda"), c["d_table"], c["d_lens"], c["scale"])
    b = paged(c, q_ptr=None)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("lens,news,page,hq,hk,d,window,sinks", [
    ([300, 47], [1, 1], 16, 8, 2, 128, 40, 4), ([300, 47], [1, 1], 16, 8, 2, 64, 40, 17), ([500], [1], 64, 8, 1, 128, 100, 3),
    ([500, 90], [20, 30], 64, 8, 2, 128, 40, 5), ([500, 90], [70, 3], 16, 2, 2, 64, 64, 0), ([900], [300], 128, 4, 1, 128, 70, 9)])
@pytest.mark.parametrize("garbage", [float("nan"), float("inf")])
def test_keys_that_no_token_sees_are_not_met(lens, news, page, hq, hk, d, window, sinks, garbage):
    # whatever stands in cached keys and values before the window of a
    # sequence's first new token (and behind the first tokens)
    c = P.make(lens, news, page, hq, hk, d, seed=2, garbage=garbage)
    for b, (n, new) in enumerate(zip(lens, news)):
        for j in range(sinks, max(sinks, n - new - window + 1)):
            for x in "kv":
                c[x][int(c["table"][b, j // page]), j % page] = garbage
    out, lse = paged(c, window, sinks, max_q=max(news))
    assert attn_last_device_error() == 0
    P.check(c, out, lse, P.reference(c, window, sinks))


def test_rows_that_see_nothing_past_32_bits_of_outputs():
    # 256 tokens of 2^18 heads of an empty sequence: 2^32 outputs of one item's rows
    hq, n = 1 << 18, 256
    kv = torch.zeros((2, 1, 16, hq, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((n, hq, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    out, lse = attn_paged_fwd(q, kv[0], kv[1], ints(0).view(1, 1), ints(0), 0.125, q_ptr=ints(0, n), out=out)
    assert attn_last_device_error() == 0
    assert not out.any() and bool((lse == -torch.inf).all())


def test_more_heads_to_a_group_than_a_row_tile_holds():
    c = P.make([200, 20], [3, 1], 32, 130, 1, 64, seed=6)
    out, lse = paged(c, 50, 2, max_q=3)
    assert attn_last_device_error() == 0
    P.check(c, out, lse, P.reference(c, 50, 2))


def test_rows_of_no_sequence_are_left_by_the_prefix_call():
    c = P.make([5, 9, 33], [2, 1, 30], 16, 8, 2, 128, seed=3, plens=[100, 40], first=[0, 1, 3], slots=[4, 0, 2], extra_tokens=2)
    T = c["q"].shape[0]
    out = torch.full((T, 8, 128), 7.0, dtype=torch.float32, device="cuda")
    lse = torch.full((8, T), 7.0, device="cuda")
    prefix(c, out=out, lse=lse)
    assert attn_last_device_error() == 0
    P.check(c, out, lse, P.reference(c))
    for x in (out[:2], out[-2:], lse[:, :2], lse[:, -2:]):
        assert torch.all(x == 7.0)


def test_prefix_bad_groups_read_nothing_out_of_range():
    c = P.make([5, 9, 33], [2, 1, 30], 16, 8, 2, 128, seed=3, plens=[100, 40], first=[0, 1, 3])
    for bad in ([0, 5, 3], [2, 1, 3], [-1, 1, 3], [0, 1, 99]):
        c["d_first"].copy_(torch.tensor(bad, dtype=torch.int32))
        prefix(c)
        assert attn_last_device_error() == B.ATTN_ERR_INVALID_ARG
    c["d_first"].copy_(torch.from_numpy(c["first"]))
    P.check(c, *prefix(c), P.reference(c))
    assert attn_last_device_error() == 0


@pytest.mark.parametrize("news", [6, 100])       # one row tile an item, two
def test_a_load_that_never_comes_ends_in_a_timeout(news, monkeypatch):
    # with ATTN_TEST_STALL_PAGED=1 every CTA leaves its second load out: the
    # bounded wait for it runs out, all roles leave their waits, tensor memory
    # is freed and the status says so; the next call is as before
    c = P.make([5000, 3000], [news, news], 64, 16, 2, 128, seed=7)
    pre = P.make([news, news], [news, news], 64, 16, 2, 128, seed=7, plens=[4000], first=[0, 2])
    a, b = paged(c), prefix(pre)
    assert attn_last_device_error() == 0
    attn_set_wait_limit_ns(50_000_000)
    monkeypatch.setenv("ATTN_TEST_STALL_PAGED", "1")
    try:
        for call in (lambda: paged(c), lambda: prefix(pre)):
            call()
            assert attn_last_device_error() == B.ATTN_ERR_TIMEOUT
    finally:
        monkeypatch.delenv("ATTN_TEST_STALL_PAGED")
        attn_set_wait_limit_ns(4_000_000_000)
    for x, y in zip(a + b, paged(c) + prefix(pre)):
        assert torch.equal(x, y)
    assert attn_last_device_error() == 0


def test_another_stream_and_a_captured_call():
    c = P.make([300, 40, 900], [1, 1, 1], 16, 8, 2, 128, seed=9)
    ref = P.reference(c, 100, 4)
    s = torch.cuda.Stream()
    out, lse = paged(c, 100, 4, q_ptr=None, stream=s)
    s.synchronize()
    P.check(c, out, lse, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out2, lse2 = paged(c, 100, 4, q_ptr=None)
    # the graph reads lengths and pages when it runs
    c["d_lens"] -= 3
    g.replay()
    torch.cuda.synchronize()
    c["lens"] = c["lens"] - 3
    P.check(c, out2, lse2, P.reference(c, 100, 4))
    assert attn_last_device_error() == 0


@pytest.mark.parametrize("news", [[1, 1, 1, 1], [3, 20, 1, 40]])
def test_a_captured_prefix_call_reads_its_arrays_when_replayed(news):
    lens = [n + 5 for n in news]
    c = P.make(lens, news, 16, 8, 2, 128, seed=11, plens=[300, 45], first=[0, 2, 4])
    s = torch.cuda.Stream()
    out, lse = prefix(c, stream=s)
    s.synchronize()
    P.check(c, out, lse, P.reference(c))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = prefix(c)
    # shorter prefixes, one of them empty, and a sequence whose first tokens see the prefix alone
    for plens, lens in (([299, 0], lens), ([17, 45], [lens[0], 0, lens[2], lens[3] - 4])):
        c["plens"], c["lens"] = np.asarray(plens, np.int32), np.asarray(lens, np.int32)
        c["d_plens"].copy_(torch.from_numpy(c["plens"]))
        c["d_lens"].copy_(torch.from_numpy(c["lens"]))
        g.replay()
        torch.cuda.synchronize()
        P.check(c, out, lse, P.reference(c))
    assert attn_last_device_error() == 0


@pytest.mark.parametrize("max_q", [1, 40])
def test_a_row_of_the_table_named_twice(max_q):
    c = P.make([70, 9, 200], [3, 3, 3], 32, 8, 2, 128, seed=5)
    c["seqs"] = np.asarray([2, 2, 0], np.int32)
    c["d_seqs"] = torch.from_numpy(c["seqs"]).cuda()
    out, lse = paged(c, 33, 2, max_q=max_q)
    assert attn_last_device_error() == 0
    P.check(c, out, lse, P.reference(c, 33, 2))


def test_many_groups_of_many_sequences():
    rng = np.random.default_rng(1)
    n = 2000
    first = np.sort(rng.integers(0, n + 1, 701)).tolist()       # empty groups among them
    c = P.make(rng.integers(0, 30, n).tolist(), [1] * n, 16, 2, 1, 64, seed=1, plens=rng.integers(0, 60, 700).tolist(), first=first)
    out, lse = prefix(c)
    assert attn_last_device_error() == 0
    P.check(c, out, lse, P.reference(c))


def test_two_calls_at_once_with_their_own_workspaces():
    c = P.make([3000, 40, 900], [1, 1, 1], 16, 8, 2, 128, seed=9)
    ref = P.reference(c)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [paged(c, q_ptr=None, stream=streams[i % 3]) for i in range(9)]
    torch.cuda.synchronize()
    for out, lse in got:
        P.check(c, out, lse, ref)


def test_prefix_calls_at_once():
    lens, news = [1000, 40, 900, 5] * 6, [1] * 24
    c = P.make(lens, news, 16, 32, 8, 128, seed=9, plens=[5000, 700], first=[0, 16, 24])
    ref = P.reference(c)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [prefix(c, stream=streams[i % 3]) for i in range(9)]
    torch.cuda.synchronize()
    P.check(c, *got[0], ref)
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    assert attn_last_device_error() == 0


@pytest.mark.parametrize("what", ["slot", "length", "negative length", "page", "negative page", "q_ptr", "q_ptr end"])
@pytest.mark.parametrize("max_q", [1, 20])
def test_bad_device_contents_are_reported_and_read_nothing(what, max_q):
    lens, news = [70, 33, 90], [2, 20, 1]
    c = P.make(lens, news, 16, 8, 2, 128, seed=8, slots=[0, 1, 2])
    ref = P.reference(c)
    if what == "slot":
        c["d_seqs"][1] = 99
    elif what == "length":
        c["d_lens"][1] = 16 * c["table"].shape[1] + 1
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
    P.check(c, out, lse, ref)
    if what in ("slot", "length", "negative length"):
        rows = slice(c["q_ptr"][1], c["q_ptr"][2])
        assert torch.all(out[rows] == 0) and torch.all(torch.isneginf(lse[:, rows]))


def test_offsets_past_32_bits():
    # pages far apart: the last one starts beyond 2^31 elements
    page, hk, d, n_pages = 256, 8, 128, 8300
    k = torch.empty((n_pages, page, hk, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = torch.tensor([[n_pages - 1, 0, n_pages - 2]], dtype=torch.int32, device="cuda")
    small = {}
    for name, x in (("k", k), ("v", v)):
        y = torch.randn((3, page, hk, d), device="cuda").bfloat16()
        for i, at in enumerate(table[0].tolist()):
            x[at] = y[i]
        small[name] = y
    assert (n_pages - 2) * page * hk * d > 2 ** 31
    q = torch.randn((1, 32, d), device="cuda").bfloat16()
    lens = torch.tensor([700], dtype=torch.int32, device="cuda")
    near = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    for n in (1, 40):
        qq = q.repeat(n, 1, 1) if n > 1 else q
        ptr = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        a = attn_paged_fwd(qq, k, v, table, lens, 0.1, q_ptr=ptr)
        b = attn_paged_fwd(qq, small["k"], small["v"], near, lens, 0.1, q_ptr=ptr)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert attn_last_device_error() == 0


def test_a_prompt_and_its_tokens_agree_with_the_windowed_slices():
    # the mask of training, through the slice list, and of serving, through
    # the cache, are one: the same rows of the same sequence
    n, h, d, window, sinks = 700, 4, 128, 100, 3
    c = P.make([n], [n], 16, h, h, d, seed=4)
    k, v = (oracle.paged.cached_rows(c[x], c["table"][0], n) for x in ("k64", "v64"))
    dev = lambda x: torch.from_numpy(x).bfloat16().cuda()  # noqa: E731
    tiles = attn_build_tiles(attn_slices_from_windows([n], window, sinks), n, n)
    out, lse = attn_fwd(c["q"], dev(k), dev(v), tiles, c["scale"])
    ref = P.reference(c, window, sinks)
    P.check(c, out, lse, ref)
    P.check(c, *paged(c, window, sinks), ref)


def test_gradients_of_the_windowed_mask():
    lengths, window, sinks, h, d = [130, 1, 300], 40, 5, 2, 64
    n = sum(lengths)
    rng = np.random.default_rng(0)
    q, k, v, do = (torch.from_numpy(rng.standard_normal((n, h, d)).astype(np.float32)).bfloat16().cuda() for _ in range(4))
    tiles = attn_build_tiles(attn_slices_from_windows(lengths, window, sinks), n, n)
    scale = d ** -0.5
    out, lse = attn_fwd(q, k, v, tiles, scale, out_dtype=torch.float32)
    got = attn_bwd(q, k, v, out, do, lse, tiles, scale)
    seen = np.zeros((n, n), bool)
    at = 0
    for m in lengths:
        i, j = np.arange(m)[:, None], np.arange(m)[None]
        seen[at:at + m, at:at + m] = (j <= i) & ((j > i - window) | (j < sinks))
        at += m
    x = [t.double().cpu().requires_grad_() for t in (q, k, v)]
    s = torch.einsum("ihd,jhd->hij", x[0], x[1]) * scale
    p = torch.softmax(s.masked_fill(~torch.from_numpy(seen), -np.inf), -1)
    torch.einsum("hij,jhd->ihd", p, x[2]).backward(do.double().cpu())
    for a, b in zip(got, x):
        e = (a.double().cpu() - b.grad).abs().max() / b.grad.abs().max()
        assert e < 0.02, e
    assert attn_last_device_error() == 0


@pytest.mark.parametrize("n,hq,hk,d", [(1025, 2, 1, 128), (1400, 4, 2, 64)])
def test_many_sequences_of_many_slabs(n, hq, hk, d):
    # above 1024 sequences each warp's ring has two slots
    rng = np.random.default_rng(n)
    c = P.make(rng.integers(0, 300, n).tolist(), [1] * n, 16, hq, hk, d, seed=n)
    for window, sinks in ((0, 0), (70, 20)):
        out, lse = paged(c, window, sinks, q_ptr=None)
        assert attn_last_device_error() == 0
        P.check(c, out, lse, P.reference(c, window, sinks))


@pytest.mark.parametrize("news", [6, 100])       # one row tile an item, two
def test_the_shortest_wait_limit_ends_a_call_in_its_result_or_in_a_timeout(news):
    # whichever role gives up first, the launch ends with its loads landed, and
    # the calls behind it are as ever
    c = P.make([5000, 3000], [news, news], 64, 16, 2, 128, seed=7)
    pre = P.make([news, news], [news, news], 64, 16, 2, 128, seed=7, plens=[4000], first=[0, 2])
    want = paged(c) + prefix(pre)
    assert attn_last_device_error() == 0
    for _ in range(20):
        attn_set_wait_limit_ns(1000)         # the least that is taken
        try:
            got = paged(c) + prefix(pre)
            status = attn_last_device_error()
        finally:
            attn_set_wait_limit_ns(4_000_000_000)
        assert status in (0, B.ATTN_ERR_TIMEOUT)
        if status == 0:
            assert all(torch.equal(x, y) for x, y in zip(want, got))
        assert all(torch.equal(x, y) for x, y in zip(want, paged(c) + prefix(pre)))
        assert attn_last_device_error() == 0


@pytest.mark.parametrize("lens,news,hq,hk,d,max_q", [
    ([3, 40], [6, 2], 4, 2, 64, 1), ([3, 0], [6, 2], 8, 1, 128, 6), ([20, 9], [50, 12], 8, 2, 128, 50), ([20, 9], [90, 100], 8, 2, 64, 100),
    ([1500, 5], [1700, 3], 4, 1, 128, 1700), ([1500, 5], [1700, 3], 4, 1, 64, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_token_that_sees_nothing_gets_zeros_whatever_the_others_see(lens, news, hq, hk, d, max_q, dtype):
    # the cached values of the sequence are infinite: its later tokens get that,
    # its first ones, which stand before its first key, zeros
    c = P.make(lens, news, 16, hq, hk, d, seed=3)
    none = np.concatenate([np.arange(new) < new - n for n, new in zip(lens, news)])
    c["v"].fill_(float("inf"))
    out, lse = paged(c, max_q=max_q, out_dtype=dtype)
    assert attn_last_device_error() == 0
    none = torch.from_numpy(none).cuda()
    assert torch.all(out[none] == 0) and torch.all(torch.isneginf(lse[:, none]))
    assert not torch.isfinite(out[~none]).any() and torch.isfinite(lse[:, ~none]).all()


def test_a_token_without_prefix_and_keys_gets_zeros_whatever_the_others_see():
    c = P.make([3, 2], [6, 7], 16, 8, 2, 128, seed=3, plens=[0, 0], first=[0, 1, 2])
    c["v"].fill_(float("inf"))
    out, lse = prefix(c, out_dtype=torch.float32)
    assert attn_last_device_error() == 0
    none = torch.tensor([True] * 3 + [False] * 3 + [True] * 5 + [False] * 2, device="cuda")
    assert torch.all(out[none] == 0) and torch.all(torch.isneginf(lse[:, none]))
    assert torch.isfinite(lse[:, ~none]).all()


@pytest.mark.parametrize("seed", range(3))
def test_hundreds_of_sequences_behind_prefixes_of_any_length(seed):
    # both passes add up the lengths of all sequences, with blocks of different sizes, to share the SMs
    rng = np.random.default_rng(seed)
    n, groups = int(rng.integers(300, 900)), int(rng.integers(1, 12))
    first = np.sort(rng.integers(0, n + 1, groups + 1)).tolist()
    c = P.make(rng.integers(0, 120, n).tolist(), [1] * n, 16, 8, 2, 64, seed=seed, plens=rng.integers(0, 3000, groups).tolist(), first=first)
    out, lse = prefix(c)
    assert attn_last_device_error() == 0
    P.check(c, out, lse, P.reference(c))
    again = prefix(c)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
