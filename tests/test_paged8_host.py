"""The cache in 8 bits and the beam search's step, on the CPU: every refusal made
before a launch."""
import ctypes

import pytest

from block_sparse_attention_slice_gb300 import beam as M
from block_sparse_attention_slice_gb300 import binding as B
from block_sparse_attention_slice_gb300 import paging as G
from test_paged_host import BAD, INV, UNS, X, Pages, Seqs

CAP = B.ATTN_ERR_CAPACITY
p = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_slice_gb300 import _build
    _build.build()
    return B.load()


class Pages8(ctypes.Structure):
    _fields_ = [("pages", Pages), ("k_scales", p), ("v_scales", p), ("scale_page_stride", ctypes.c_int64),
                ("scale_token_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64), ("format", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def _args(**kw):
    pages8 = Pages8(Pages(4096, 4096, 10, 16, 2, 128, 16 * 256, 256, 128), 4096, 4096, 32, 2, 1, 0, 0)
    a = dict(q=X, q_ptr=X, n_tokens=5, max_q=2, hq=4, scale=1.0, window=0, sinks=0, out=X, out_dtype=0, lse=X, ws=X, ws_bytes=1 << 40,
             group_ptr=X, pages8=pages8, seqs=Seqs(4096, 4096, None, 4, 3, 4, 3, 0), pre=Seqs(4096, 4096, None, 4, 1, 4, 1, 0))
    for name, value in kw.items():
        of, _, field = name.partition("__")
        if of == "pages" and field:
            setattr(pages8.pages, field, value)
        elif field:
            setattr(a[of], field, value)
        elif name == "pages":
            a["pages8"] = value
        else:
            a[name] = value
    return a


ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731


def _attend(lib, a, prefix):
    if prefix:
        return lib.attn_prefix8_fwd(a["q"], a["q_ptr"], a["n_tokens"], a["max_q"], a["hq"], ref(a["pages8"]), ref(a["pre"]), a["group_ptr"],
                                    ref(a["seqs"]), a["scale"], a["out"], a["out_dtype"], a["lse"], a["ws"], a["ws_bytes"], None)
    return lib.attn_paged8_fwd(a["q"], a["q_ptr"], a["n_tokens"], a["max_q"], a["hq"], ref(a["pages8"]), ref(a["seqs"]), a["scale"],
                               a["window"], a["sinks"], a["out"], a["out_dtype"], a["lse"], a["ws"], a["ws_bytes"], None)


BAD8 = [({"pages8__k_scales": None}, INV), ({"pages8__v_scales": None}, INV), ({"pages8__format": 2}, INV), ({"pages8__format": -1}, INV),
        ({"pages__page_stride": 4104}, UNS), ({"pages__token_stride": 264}, UNS), ({"pages__head_stride": 8}, UNS),
        ({"pages8__k_scales": 4098}, UNS), ({"pages8__v_scales": 4097}, UNS), ({"pages8__scale_page_stride": -1}, UNS),
        ({"pages8__scale_token_stride": -1}, UNS), ({"pages8__scale_head_stride": -2}, UNS)]


@pytest.mark.parametrize("change,code", BAD + BAD8, ids=[str(i) for i in range(len(BAD + BAD8))])
@pytest.mark.parametrize("prefix", [False, True])
def test_refusals(lib, change, code, prefix):
    assert _attend(lib, _args(**change), prefix) == code


@pytest.mark.parametrize("prefix", [False, True])
def test_empty_batches_do_nothing(lib, prefix):
    assert _attend(lib, _args(n_tokens=0), prefix) == B.ATTN_OK
    assert _attend(lib, _args(n_tokens=0, q=None, out=None, lse=None, ws=None, q_ptr=None, seqs__n_seqs=0), prefix) == B.ATTN_OK


@pytest.mark.parametrize("prefix", [False, True])
def test_outputs_on_top_of_inputs_are_refused(lib, prefix):
    # q and a bf16 out: 5120 bytes; pages: 9 x 4096 + 15 x 256 + 128 + 128 = 40960; scales: (9 x 32 + 15 x 2 + 1 + 1) x 4 = 1280
    clear = dict(q=p(1 << 20), out=p((1 << 20) + 5120), ws=p(1 << 30))
    assert _attend(lib, _args(**clear), prefix) not in (INV, UNS)
    for free in (dict(out=p(4096 + 40960)), dict(pages8__k_scales=(1 << 20) + 10240), dict(pages8__v_scales=(1 << 20) + 5120 - 1280)):
        if "out" not in free:
            free["q"] = p(1 << 24)
        assert _attend(lib, _args(**{**clear, **free}), prefix) not in (INV, UNS), free
    for bad in (dict(out=p(1 << 20)), dict(out=p(4096 + 40944)), dict(pages__v=(1 << 20) + 5120 + 5104),
                dict(pages8__k_scales=(1 << 20) + 10236), dict(pages8__v_scales=(1 << 20) + 5120 - 1276)):
        assert _attend(lib, _args(**{**clear, **bad}), prefix) == INV, bad


def _write(lib, k=X, v=X, q_ptr=X, n=5, ts=256, hs=128, **kw):
    a = _args(**kw)
    return lib.attn_cache8_write(ref(a["pages8"]), ref(a["seqs"]), q_ptr, k, v, n, ts, hs, None)


def _read(lib, k=X, v=X, q_ptr=X, n=5, dtype=0, bits8=True, **kw):
    a = _args(**kw)
    if bits8:
        return lib.attn_cache8_read(ref(a["pages8"]), ref(a["seqs"]), q_ptr, n, k, v, dtype, None)
    return lib.attn_cache_read(ref(a["pages8"] and a["pages8"].pages), ref(a["seqs"]), q_ptr, n, k, v, dtype, None)


TOKENS = [({"k": None}, INV), ({"v": None}, INV), ({"q_ptr": None}, INV), ({"n": -1}, INV), ({"pages__hk": 0}, INV), ({"seqs__table": None}, INV),
          ({"pages": None}, INV), ({"seqs": None}, INV), ({"seqs__seq_lens": None}, INV), ({"k": p(4104)}, UNS), ({"v": p(4100)}, UNS),
          ({"pages__page_size": 20}, UNS), ({"n": (1 << 30) + 1}, UNS), ({"pages__d": 32}, UNS), ({"pages__hk": 1025}, UNS),
          ({"seqs__n_seqs": 4097, "seqs__seqs": 4096}, UNS)]


@pytest.mark.parametrize("change,code", TOKENS, ids=[str(i) for i in range(len(TOKENS))])
def test_refusals_of_tokens(lib, change, code):
    assert _write(lib, **change) == code
    assert _read(lib, **change) == code
    assert _read(lib, bits8=False, **change) == code


def test_refusals_of_writes_and_reads(lib):
    for change, code in BAD8:
        assert _write(lib, **change) == code
        assert _read(lib, **change) == code
    for bad in ({"ts": 100}, {"hs": 12}, {"ts": -256}, {"pages__page_stride": 0}, {"pages__token_stride": 0}, {"pages__head_stride": 0},
                {"pages8__scale_page_stride": 0}, {"pages8__scale_token_stride": 0}, {"pages8__scale_head_stride": 0}):
        assert _write(lib, **bad) == UNS      # places seen as several are fine to read, not to write
    for dtype in (-1, 2):
        assert _read(lib, dtype=dtype) == INV and _read(lib, dtype=dtype, bits8=False) == INV
    for nothing in (dict(n=0), dict(n=0, k=None, v=None), dict(n=0, q_ptr=None, seqs__n_seqs=0)):
        assert _write(lib, **nothing) == _read(lib, **nothing) == _read(lib, bits8=False, **nothing) == B.ATTN_OK


def _select(lib, logits=X, dtype=1, stride=100, groups=2, beams=4, vocab=100, scores=X, done=X, eos=3, slots=X, keep=4, os=X, op=X, ot=X,
            od=X, src=X, ws=X, ws_bytes=1 << 40):
    return lib.attn_beam_select(logits, dtype, stride, groups, beams, vocab, scores, done, eos, slots, keep, os, op, ot, od, src, ws, ws_bytes,
                                None)


SELECT = [({"logits": None}, INV), ({"scores": None}, INV), ({"os": None}, INV), ({"op": None}, INV), ({"ot": None}, INV), ({"ws": None}, INV),
          ({"dtype": 2}, INV), ({"dtype": -1}, INV), ({"stride": 99}, INV), ({"groups": -1}, INV), ({"beams": 0}, INV), ({"vocab": 0}, INV),
          ({"keep": 0}, INV), ({"vocab": 1, "eos": 0, "keep": 5}, INV), ({"eos": 100}, INV), ({"eos": -2}, INV), ({"eos": -1}, INV),
          ({"beams": 65}, UNS), ({"keep": 65}, UNS), ({"groups": 1 << 22}, UNS), ({"vocab": (1 << 30) + 1, "stride": 1 << 31}, UNS),
          ({"logits": p(4098)}, UNS), ({"logits": p(4097), "dtype": 0}, UNS), ({"scores": p(4098)}, UNS), ({"slots": p(4097)}, UNS),
          ({"os": p(4097)}, UNS), ({"op": p(4098)}, UNS), ({"ot": p(4099)}, UNS), ({"src": p(4097)}, UNS), ({"ws": p(4104)}, UNS)]


@pytest.mark.parametrize("change,code", SELECT, ids=[str(i) for i in range(len(SELECT))])
def test_refusals_of_select(lib, change, code):
    assert _select(lib, **change) == code


def test_select_without_prompts(lib):
    assert _select(lib, groups=0, logits=None, scores=None, os=None, op=None, ot=None, ws=None) == B.ATTN_OK
    assert _select(lib, groups=0, keep=0) == INV
    assert lib.attn_beam_workspace_bytes(1, 4, 100, 4, None) == INV


def _reorder(lib, states=(4096, 8192), row=(64, 64), stride=(64, 80), n=None, parents=X, groups=2, beams=4):
    k = len(states)
    arrays = (p * k)(*states), (ctypes.c_int64 * k)(*row), (ctypes.c_int64 * k)(*stride)
    return lib.attn_beam_reorder(*arrays, k if n is None else n, parents, groups, beams, None)


def test_refusals_of_reorder(lib):
    for bad in (dict(n=-1), dict(groups=-1), dict(beams=0), dict(parents=None), dict(states=(4096, None)), dict(row=(64, -1)), dict(row=(65, 64)),
                dict(states=(4096, 4096))):
        assert _reorder(lib, **bad) == INV, bad
    assert lib.attn_beam_reorder(None, None, None, 1, X, 1, 2, None) == INV
    for bad in (dict(beams=65), dict(groups=1 << 22), dict(parents=p(4098)), dict(states=(4096,) * 65, row=(64,) * 65, stride=(64,) * 65)):
        assert _reorder(lib, **bad) == UNS, bad
    assert _reorder(lib, groups=0, parents=None) == B.ATTN_OK
    assert _reorder(lib, n=0) == B.ATTN_OK
    assert _reorder(lib, states=(None, None), row=(0, 0)) == B.ATTN_OK


def test_binding_refuses_wrong_tensors(lib):
    import torch
    codes = torch.zeros((4, 16, 2, 64), dtype=torch.int8)
    scales = torch.zeros((4, 16, 2))
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    both = dict(k_scales=scales, v_scales=scales)
    for pages, kw in ((codes, both), (codes, {}), (codes, dict(k_scales=scales)), (codes, dict(k_scales=scales, v_scales=scales[:, :, :1])),
                      (k, both), (codes.view(torch.uint8), both), (codes, dict(k_scales=scales.double(), v_scales=scales.double()))):
        for call in (lambda: G.attn_paged_fwd(q, pages, pages, i[None], i, 1.0, **kw),
                     lambda: G.attn_prefix_fwd(q, pages, pages, i[None], i, i, i[None], i, 1.0, **kw),
                     lambda: G.attn_cache_write(pages, pages, q, q, i[None], i, **kw),
                     lambda: G.attn_cache_read(pages, pages, i[None], i, 1, **kw)):
            with pytest.raises(ValueError):
                call()
    with pytest.raises(TypeError):
        G.attn_cache_read(None, k, i[None], i, 1)
    x = torch.zeros((2, 8))
    for call in (lambda: M.attn_beam_select(x, x[:, :1]), lambda: M.attn_beam_reorder([x], torch.zeros((1, 2), dtype=torch.int32))):
        with pytest.raises(ValueError):      # not on a GPU
            call()
    for call in (lambda: M.attn_beam_select(None, x), lambda: M.attn_beam_reorder([x], None)):
        with pytest.raises(TypeError):
            call()
