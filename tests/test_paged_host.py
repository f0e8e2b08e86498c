"""Attention over a paged cache, on the CPU: the oracle against brute force,
the windowed slice list, and every refusal made before a launch."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

import oracle
from block_sparse_attention_slice_gb300 import binding as B
from block_sparse_attention_slice_gb300 import paging as G


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_slice_gb300 import _build
    _build.build()
    return B.load()


@pytest.mark.parametrize("lengths", [[], [0], [1], [7, 0, 30], [64, 33, 100]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 5), (1, 0), (1, 1), (4, 0), (4, 3), (10, 40), (200, 2), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windowed_slices_are_the_mask(lib, lengths, window, sinks):
    got = G.attn_slices_from_windows(lengths, window, sinks)
    n = sum(lengths)
    want = np.zeros((n, n), bool)
    at = 0
    for m in lengths:
        for i in range(m):
            for j in range(i + 1):
                want[at + i, at + j] = window == 0 or j > i - window or j < sinks
        at += m
    if n:
        assert np.array_equal(oracle.mask_rows(got, np.arange(n), n), want)
    assert len(got) <= 3 * len(lengths)
    r = [x for x in got.tolist()]
    for i, a in enumerate(r):
        for b in r[i + 1:]:
            assert not (a[0] < b[1] and b[0] < a[1] and a[2] < b[3] and b[2] < a[3])


def test_windowed_slices_refusals(lib):
    for args in (([-1], 1, 0), ([3], -1, 0), ([3], 1, -1), ([2 ** 31 - 1, 1], 1, 0)):
        with pytest.raises(B.AttnError) as e:
            G.attn_slices_from_windows(*args)
        assert e.value.code == B.ATTN_ERR_INVALID_ARG
    n = ctypes.c_int(0)
    a = (ctypes.c_int32 * 1)(100)
    assert lib.attn_slices_from_windows(a, 1, 4, 1, None, 0, ctypes.byref(n)) == B.ATTN_ERR_CAPACITY
    assert n.value == 3
    assert lib.attn_slices_from_windows(a, 1, 4, 1, None, 0, None) == B.ATTN_ERR_INVALID_ARG


def test_oracle_paged_is_the_dense_oracle():
    rng = np.random.default_rng(0)
    n, H, hk, d, page = 37, 4, 2, 8, 16
    k, v = rng.standard_normal((2, 5, page, hk, d))
    table = np.array([[3, 0, 4]])
    q = rng.standard_normal((n, H, d))
    O, lse, _, _ = oracle.oracle_paged(q, k, v, table, [n], [0, n], 0.3, 7, 2)
    kk, vv = (oracle.paged.cached_rows(x, table[0], n) for x in (k, v))
    i, j = np.arange(n)[:, None], np.arange(n)
    mask = (j <= i) & ((j > i - 7) | (j < 2))
    ref = oracle.oracle_attention(q, kk, vv, 0.3, lambda r: mask[r])
    for h in range(H):
        assert np.allclose(O[:, h], ref[h][1]) and np.allclose(lse[h], ref[h][2])
    # the first 20 tokens as a prefix of the others
    pre = (table, [20], [0, 1])
    rest = np.array([[1, 2]])
    k2, v2 = k.copy(), v.copy()
    for x, y in ((k2, kk), (v2, vv)):
        for u in range(n - 20):
            x[rest[0, u // page], u % page] = y[20 + u]
    O2, l2, _, _ = oracle.oracle_paged(q[20:], k2, v2, rest, [n - 20], [0, n - 20], 0.3, prefix=pre)
    O1, l1, _, _ = oracle.oracle_paged(q, k, v, table, [n], [0, n], 0.3)
    assert np.allclose(O2, O1[20:]) and np.allclose(l2, l1[:, 20:])


class Pages(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("hk", ctypes.c_int32), ("d", ctypes.c_int32), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class Seqs(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("seqs", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("n_slots", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("n_seqs", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Cache(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("refs", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("n_slots", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32)]


X = ctypes.c_void_p(4096)      # an aligned address that no refused call reads


def _args(**kw):
    pages = Pages(4096, 4096, 10, 16, 2, 128, 16 * 256, 256, 128)
    seqs = Seqs(4096, 4096, None, 4, 3, 4, 3, 0)
    pre = Seqs(4096, 4096, None, 4, 1, 4, 1, 0)
    a = dict(q=X, q_ptr=X, n_tokens=5, max_q=2, hq=4, scale=1.0, window=0, sinks=0, out=X, out_dtype=0, lse=X, ws=X, ws_bytes=1 << 40,
             group_ptr=X, pages=pages, seqs=seqs, pre=pre)
    for name, value in kw.items():
        if "__" in name:
            setattr(a[name.split("__")[0]], name.split("__")[1], value)
        else:
            a[name] = value
    return a


def _call(lib, a, prefix):
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    if prefix:
        return lib.attn_prefix_fwd(a["q"], a["q_ptr"], a["n_tokens"], a["max_q"], a["hq"], ref(a["pages"]), ref(a["pre"]), a["group_ptr"],
                                   ref(a["seqs"]), a["scale"], a["out"], a["out_dtype"], a["lse"], a["ws"], a["ws_bytes"], None)
    return lib.attn_paged_fwd(a["q"], a["q_ptr"], a["n_tokens"], a["max_q"], a["hq"], ref(a["pages"]), ref(a["seqs"]), a["scale"],
                              a["window"], a["sinks"], a["out"], a["out_dtype"], a["lse"], a["ws"], a["ws_bytes"], None)


INV, UNS = B.ATTN_ERR_INVALID_ARG, B.ATTN_ERR_UNSUPPORTED
BAD = [({"q": None}, INV), ({"out": None}, INV), ({"lse": None}, INV), ({"ws": None}, INV), ({"pages": None}, INV), ({"seqs": None}, INV),
       ({"q_ptr": None}, INV), ({"n_tokens": -1}, INV), ({"max_q": 0}, INV), ({"hq": 0}, INV), ({"hq": 3}, INV), ({"scale": 0.0}, INV),
       ({"scale": -1.0}, INV), ({"scale": float("nan")}, INV), ({"scale": float("inf")}, INV), ({"out_dtype": 2}, INV),
       ({"pages__k": None}, INV), ({"pages__v": None}, INV), ({"pages__n_pages": 0}, INV), ({"pages__hk": 0}, INV), ({"pages__d": 96}, UNS),
       ({"pages__page_size": 8}, UNS), ({"pages__page_size": 48}, UNS), ({"pages__page_size": 0}, UNS), ({"pages__k": 4098}, UNS),
       ({"pages__page_stride": 4100}, UNS), ({"pages__token_stride": 257}, UNS), ({"pages__head_stride": -128}, UNS),
       ({"seqs__table": None}, INV), ({"seqs__seq_lens": None}, INV), ({"seqs__n_seqs": -1}, INV), ({"seqs__n_slots": 2}, INV),
       ({"seqs__table_stride": 3}, INV), ({"seqs__max_pages": -1}, INV), ({"q": ctypes.c_void_p(4098)}, UNS),
       ({"out": ctypes.c_void_p(4104)}, UNS), ({"ws": ctypes.c_void_p(4104)}, UNS)]


@pytest.mark.parametrize("change,code", BAD, ids=[str(i) for i in range(len(BAD))])
@pytest.mark.parametrize("prefix", [False, True])
def test_refusals(lib, change, code, prefix):
    assert _call(lib, _args(**change), prefix) == code


def test_refusals_of_one_call(lib):
    for change in ({"window": -1}, {"sinks": -1}):
        assert _call(lib, _args(**change), False) == INV
    for change in ({"group_ptr": None}, {"pre": None}, {"pre__table": None}, {"pre__table_stride": 1}, {"pre__n_slots": 0}):
        assert _call(lib, _args(**change), True) == INV
    for prefix in (False, True):
        a = _args()
        a["seqs"].seqs, a["seqs"].n_seqs = 4096, 4097
        assert _call(lib, a, prefix) == UNS
        a = _args()
        a["seqs"].max_pages = a["seqs"].table_stride = (1 << 26) + 1
        assert _call(lib, a, prefix) == UNS
        a = _args()
        a["seqs"].seqs, a["seqs"].n_seqs, a["seqs"].max_pages, a["seqs"].table_stride = 4096, 4096, 1 << 21, 1 << 21
        assert _call(lib, a, prefix) == UNS
        assert _call(lib, _args(n_tokens=1 << 29, hq=4), prefix) == UNS
        # an empty batch is no error and launches nothing
        assert _call(lib, _args(n_tokens=0), prefix) == B.ATTN_OK
        a = _args(n_tokens=0, q=None, out=None, lse=None, ws=None, q_ptr=None)
        a["seqs"].n_seqs = 0
        assert _call(lib, a, prefix) == B.ATTN_OK


def test_binding_refuses_wrong_tensors(lib):
    import torch
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    for bad in ((q, k, k), (q, k, k[:, :, :1]), (q, k.float(), k.float()), (q, k[0], k[0])):        # not on a GPU, or worse
        with pytest.raises(ValueError):
            G.attn_paged_fwd(*bad, i[None], i, 1.0)
        with pytest.raises(ValueError):
            G.attn_prefix_fwd(*bad, i[None], i, i, i[None], i, 1.0)
    with pytest.raises(TypeError):
        G.attn_paged_fwd(q, None, k, i[None], i, 1.0)
    for call in (lambda: G.attn_cache_free(i[None], i, i, i, 16), lambda: G.attn_cache_extend(i[None], i, i, i, i, 16),
                 lambda: G.attn_cache_trim(i[None], i, i, 16, 1), lambda: G.attn_cache_fork(i[None], i, i, i, i, 16),
                 lambda: G.attn_cache_compact(i[None], i, i, 16), lambda: G.attn_cache_copy_pages([k], i),
                 lambda: G.attn_cache_write(k, k, q, q, i[None], i)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        G.attn_cache_copy_pages(7, i)


def _cache(**kw):
    c = Cache(4096, 4096, 4096, 6, 5, 6, 40, 16)
    for name, value in kw.items():
        setattr(c, name, value)
    return ctypes.byref(c)


CACHE_BAD = [({"table": None}, INV), ({"seq_lens": None}, INV), ({"refs": None}, INV), ({"n_slots": 0}, INV), ({"max_pages": 0}, INV),
             ({"n_pages": 0}, INV), ({"table_stride": 5}, INV), ({"page_size": 8}, UNS), ({"page_size": 24}, UNS), ({"n_slots": 16385}, UNS),
             ({"max_pages": 1 << 27, "table_stride": 1 << 27}, UNS), ({"n_pages": (1 << 30) + 1}, UNS),
             ({"n_slots": 16384, "max_pages": 1 << 20, "table_stride": 1 << 20}, UNS)]


@pytest.mark.parametrize("change,code", CACHE_BAD, ids=[str(i) for i in range(len(CACHE_BAD))])
def test_cache_refusals(lib, change, code):
    n = ctypes.c_size_t(0)
    c = _cache(**change)
    assert lib.attn_cache_extend(c, X, X, 1, None) == code
    assert lib.attn_cache_free(c, X, 1, None) == code
    assert lib.attn_cache_trim(c, X, 1, 4, 0, None) == code
    assert lib.attn_cache_fork(c, X, X, 1, X, 1, X, 1 << 40, None) == code
    assert lib.attn_cache_compact(c, X, 1, X, 1 << 40, None) == code
    assert lib.attn_cache_workspace_bytes(c, 1, ctypes.byref(n)) == code


def test_cache_list_refusals(lib):
    n = ctypes.c_size_t(0)
    CAP = B.ATTN_ERR_CAPACITY
    for count, code in ((-1, INV), (6, INV), (4097, UNS)):     # more rows than the table has: one would be named twice
        assert lib.attn_cache_extend(_cache(), X, X, count, None) == code
        assert lib.attn_cache_free(_cache(), X, count, None) == code
        assert lib.attn_cache_trim(_cache(), X, count, 4, 0, None) == code
        assert lib.attn_cache_fork(_cache(), X, X, count, X, 9, X, 1 << 40, None) == code
    assert lib.attn_cache_extend(_cache(), None, X, 1, None) == INV
    assert lib.attn_cache_extend(_cache(), X, None, 1, None) == INV
    assert lib.attn_cache_free(_cache(), None, 1, None) == INV
    assert lib.attn_cache_trim(_cache(), None, 4, 4, 0, None) == INV       # every row, or a list
    assert lib.attn_cache_trim(_cache(), X, 4, 0, 0, None) == INV
    assert lib.attn_cache_trim(_cache(), X, 4, 4, -1, None) == INV
    assert lib.attn_cache_fork(_cache(), X, X, 2, None, 2, X, 1 << 40, None) == INV
    assert lib.attn_cache_fork(_cache(), X, X, 2, X, -1, X, 1 << 40, None) == INV
    assert lib.attn_cache_fork(_cache(), X, X, 2, X, 2, None, 1 << 40, None) == INV
    assert lib.attn_cache_fork(_cache(), X, X, 2, X, 2, ctypes.c_void_p(4097), 1 << 40, None) == UNS
    assert lib.attn_cache_workspace_bytes(_cache(), 2, ctypes.byref(n)) == B.ATTN_OK
    assert lib.attn_cache_fork(_cache(), X, X, 2, X, 2, X, 4 * 2 * 7 - 1, None) == CAP and n.value >= 4 * 2 * 7
    assert lib.attn_cache_compact(_cache(), None, 1, X, 1 << 40, None) == INV
    assert lib.attn_cache_compact(_cache(), X, 1, None, 1 << 40, None) == INV
    assert lib.attn_cache_compact(_cache(), X, 1, X, 4 * 40 - 1, None) == CAP and n.value >= 4 * 40
    assert lib.attn_cache_workspace_bytes(_cache(), -1, ctypes.byref(n)) == INV
    assert lib.attn_cache_extend(_cache(), X, X, 0, None) == B.ATTN_OK
    assert lib.attn_cache_free(_cache(), X, 0, None) == B.ATTN_OK


def test_copy_and_write_refusals(lib):
    pools = (ctypes.c_void_p * 2)(4096, 8192)
    copy = lambda p=pools, n=2, size=64, stride=64, pages=4, c=X, cap=3: lib.attn_cache_copy_pages(p, n, size, stride, pages, c, cap, None)  # noqa: E731
    assert copy(n=0) == B.ATTN_OK and copy(cap=0) == B.ATTN_OK
    for bad in ({"p": None}, {"n": -1}, {"size": 0}, {"stride": 48}, {"pages": 0}, {"c": None}, {"cap": -1}, {"p": (ctypes.c_void_p * 2)(4096, None)}):
        assert copy(**bad) == INV
    for bad in ({"n": 257}, {"size": 60}, {"stride": 72}, {"size": 1 << 31, "stride": 1 << 31}, {"p": (ctypes.c_void_p * 2)(4096, 4104)}):
        assert copy(**bad) == UNS

    def write(k=X, v=X, q_ptr=X, n=5, ts=256, hs=128, **kw):
        a = _args(**kw)
        return lib.attn_cache_write(ctypes.byref(a["pages"]), ctypes.byref(a["seqs"]), q_ptr, k, v, n, ts, hs, None)
    assert write(n=0) == B.ATTN_OK
    for bad in ({"k": None}, {"v": None}, {"q_ptr": None}, {"n": -1}, {"pages__hk": 0}, {"seqs__table": None}):
        assert write(**bad) == INV
    for bad in ({"k": ctypes.c_void_p(4104)}, {"ts": 100}, {"hs": 12}, {"ts": -256}, {"pages__page_size": 20}):
        assert write(**bad) == UNS


def test_write_refuses_places_seen_as_several(lib):
    for bad in ({"pages__page_stride": 0}, {"pages__token_stride": 0}, {"pages__head_stride": 0}):
        a = _args(**bad)
        assert lib.attn_cache_write(ctypes.byref(a["pages"]), ctypes.byref(a["seqs"]), X, X, X, 5, 256, 128, None) == UNS
    a = _args()
    assert lib.attn_cache_write(ctypes.byref(a["pages"]), ctypes.byref(a["seqs"]), X, X, X, (1 << 30) + 1, 0, 128, None) == UNS


@pytest.mark.parametrize("prefix", [False, True])
def test_outputs_on_top_of_inputs_are_refused(lib, prefix):
    # q: 5 x 4 x 128 bf16 = 5120 bytes; pages: (9 x 4096 + 15 x 256 + 128 + 128) x 2 = 81920 bytes
    p = lambda at: ctypes.c_void_p(at)  # noqa: E731
    clear = dict(q=p(1 << 20), out=p((1 << 20) + 5120), ws=p(1 << 30))
    assert _call(lib, _args(**clear), prefix) not in (INV, UNS)
    for bad in (dict(q=p(1 << 20), out=p(1 << 20)), dict(q=p(1 << 20), out=p((1 << 20) + 5104)),
                dict(q=p(1 << 20), out=p((1 << 20) - 10224), out_dtype=1), dict(q=p(1 << 20), out=p(4096 + 81904)),
                dict(q=p(1 << 20), out=p(1 << 24), pages__v=(1 << 24) - 16)):
        assert _call(lib, _args(**{**clear, **bad}), prefix) == INV


@pytest.mark.parametrize("args", [([100], 2 ** 32 + 3, 0), ([100], 2 ** 31, 0), ([100], 4, 2 ** 32), ([100], -2 ** 32 + 4, 0), ([100], 4, 2 ** 64),
                                  (np.array([2 ** 32 + 5]), 4, 0), (np.array([7, 2 ** 31]), 4, 0), (np.array([-2 ** 32 + 5]), 4, 0),
                                  (np.array([2 ** 63 + 5], np.uint64), 4, 0), ([2 ** 70], 4, 0), ([7.5], 4, 0), ([7], 4.5, 0),
                                  ([float("nan")], 4, 0), ([7], float("inf"), 0)], ids=str)
def test_windowed_slices_refuse_what_32_bits_do_not_hold(lib, args):
    with pytest.raises((ValueError, OverflowError)):
        G.attn_slices_from_windows(*args)


def test_windowed_slices_take_whole_numbers_of_any_type(lib):
    want = G.attn_slices_from_windows([70, 9], 33, 2)
    for lengths, window, sinks in ((np.array([70, 9], np.int64), 33, 2), (np.array([70, 9], np.uint8), np.int64(33), np.int8(2)),
                                   ([70.0, 9.0], 33.0, 2), ((70, 9), 33, 2)):
        assert np.array_equal(G.attn_slices_from_windows(lengths, window, sinks), want)
    import torch
    assert np.array_equal(G.attn_slices_from_windows(torch.tensor([70, 9]), torch.tensor(33), 2), want)


def test_the_package_and_its_host_functions_do_without_torch(lib):
    # PyTorch is needed where tensors are taken, not to import the package or to make a slice list
    code = ("import sys; sys.modules['torch'] = None\n"
            "import block_sparse_attention_slice_gb300 as attn\n"
            "attn.load()\n"
            "print(len(attn.attn_slices_from_windows([70, 9], 33, 2)), len(attn.attn_slices_from_block_grid([[1, 0], [1, 2]], 64, 64)))\n")
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                          cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert done.returncode == 0, done.stderr
    assert done.stdout.split() == [str(len(G.attn_slices_from_windows([70, 9], 33, 2))), "3"]
