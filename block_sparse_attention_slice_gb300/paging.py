"""Thin Python binding of the C ABI in ``include/attn_paged.h``: attention
over a paged key/value cache and the pages of that cache.

Argument marshalling only, as in ``binding.py``: the computation runs in the
CUDA kernels of ``libattn_slice.so``, and there is no fallback.  Index arrays
(tables, lengths, lists) are int32 CUDA tensors and are checked by the kernels;
what they find is reported by ``attn_last_device_error``.

A call runs on its tensors' device, on ``stream`` or that device's current
stream.
"""
from __future__ import annotations

import ctypes
from typing import Sequence

import numpy as np

from . import binding as B


class AttnPages(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("hk", ctypes.c_int32), ("d", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class AttnSeqs(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("seqs", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("n_slots", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("n_seqs", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def _ints(device, **arrays):
    """int32 vectors on `device`, contiguous; None stays None."""
    import torch
    for name, x in arrays.items():
        if x is None:
            continue
        if x.dtype != torch.int32 or x.dim() != 1 or x.device != device or (x.numel() > 1 and x.stride(0) != 1):
            raise ValueError(f"{name} must be a contiguous int32 vector on {device}")


def _pages(k, v):
    import torch
    if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.stride(3) != 1:
        raise ValueError("k_pages and v_pages must be [n_pages, page_size, H_k, d], alike in strides, d contiguous")
    if k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16 or not k.is_cuda or v.device != k.device:
        raise ValueError("k_pages and v_pages must be bf16 tensors on one CUDA device")
    n, page, hk, d = k.shape
    sp, st, sh, _ = k.stride()
    return AttnPages(k.data_ptr(), v.data_ptr(), n, page, hk, d, sp, st, sh)


def _seqs(device, table, seq_lens, seqs, what=""):
    import torch
    if table.dtype != torch.int32 or table.dim() != 2 or table.device != device or \
            (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"{what}table must be int32 [n_slots, max_pages] on {device}, rows contiguous")
    _ints(device, **{what + "seq_lens": seq_lens, what + "seqs": seqs})
    if seq_lens.shape[0] != table.shape[0]:
        raise ValueError(f"{what}table and {what}seq_lens must have one row a slot")
    n, width = table.shape
    stride = table.stride(0) if n > 1 else max(width, table.stride(0))
    return AttnSeqs(table.data_ptr(), seq_lens.data_ptr(), None if seqs is None else seqs.data_ptr(), stride,
                    n, width, n if seqs is None else seqs.shape[0], 0)


class AttnCache(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("n_slots", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32)]


def _cache(table, seq_lens, refs, page_size):
    s = _seqs(table.device, table, seq_lens, None)
    if not table.is_cuda:
        raise ValueError("the cache's arrays must be CUDA tensors")
    _ints(table.device, refs=refs)
    return AttnCache(s.table, s.seq_lens, refs.data_ptr(), s.table_stride, s.n_slots, s.max_pages, refs.shape[0],
                     int(page_size))


def _lists(device, a, b=None, names=("seqs", "counts")):
    _ints(device, **{names[0]: a, names[1]: b})
    if b is not None and a.shape != b.shape:
        raise ValueError(f"{names[0]} and {names[1]} must be of one length")


class _On:
    """Makes a tensor's device the current one for a call, where it is not."""

    def __init__(self, device):
        import torch
        self.guard = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *a):
        if self.guard is not None:
            self.guard.__exit__(*a)


def _borrowed(stream, *tensors):
    """Tensors allocated here on the current stream and used on another one."""
    import torch
    if stream is not None and stream != torch.cuda.current_stream():
        stream.wait_stream(torch.cuda.current_stream())
        for x in tensors:
            x.record_stream(stream)


def _attend(name, q, pages, seqs, device, scale, q_ptr, max_q, out, lse, out_dtype, ws, stream, call, prefix):
    import torch
    if q.dtype != torch.bfloat16 or q.dim() != 3 or q.device != device or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous bf16 [n_tokens, H, d] tensor on {device}")
    t, hq, d = q.shape
    if d != pages.d:
        raise ValueError("q and the pages must have one head dim")
    _ints(device, q_ptr=q_ptr)
    if q_ptr is not None and q_ptr.shape[0] != seqs.n_seqs + 1:
        raise ValueError("q_ptr must have one entry a sequence and one more")
    made = []
    with _On(device):
        if out is None:
            out = torch.empty((t, hq, d), dtype=out_dtype or torch.bfloat16, device=device)
            made.append(out)
        elif out.shape != q.shape or out.device != device or not out.is_contiguous() or \
                out.dtype not in (torch.bfloat16, torch.float32) or out_dtype not in (None, out.dtype):
            raise ValueError("out must be a contiguous bf16 or f32 tensor like q")
        if lse is None:
            lse = torch.empty((hq, t), dtype=torch.float32, device=device)
            made.append(lse)
        elif lse.shape != (hq, t) or lse.dtype != torch.float32 or lse.device != device or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous f32 [H, n_tokens] tensor")
        if ws is None:
            nb = ctypes.c_size_t(0)
            B._check(B.load().attn_paged_workspace_bytes(t, hq, d, prefix, ctypes.byref(nb)), "attn_paged_workspace_bytes")
            ws = torch.empty(nb.value, dtype=torch.uint8, device=device)
            made.append(ws)
        elif ws.device != device or not ws.is_contiguous():
            raise ValueError("ws must be a contiguous tensor on the queries' device")
        if stream is not None:
            _borrowed(stream, *made)
        code = B.ATTN_DTYPE_F32 if out.dtype == torch.float32 else B.ATTN_DTYPE_BF16
        if max_q is None:
            max_q = 1 if q_ptr is None else max(1, t)
        B._check(call(q.data_ptr(), None if q_ptr is None else q_ptr.data_ptr(), t, int(max_q), hq, pages, seqs,
                      float(scale), out.data_ptr(), code, lse.data_ptr(), ws.data_ptr(),
                      ws.numel() * ws.element_size(), B._stream_ptr(stream)), name)
    return out, lse


def attn_paged_fwd(q, k_pages, v_pages, table, seq_lens, scale: float, q_ptr=None, max_q=None, window: int = 0,
                   sinks: int = 0, seqs=None, out=None, lse=None, out_dtype=None, ws=None, stream=None):
    """O, lse of each sequence's newest tokens over its cached keys.

    q [n_tokens,H,d] bf16; k_pages/v_pages [n_pages,page_size,H_k,d] bf16;
    table int32 [n_slots,max_pages]; seq_lens int32 [n_slots] (the new tokens,
    whose keys are cached already, included); q_ptr int32 [n_seqs+1] (None:
    one token a sequence); seqs int32 [n_seqs] table rows (None: all, in
    order).  A token at position i sees keys j <= i with j > i - window or
    j < sinks (window 0: all).  ``max_q`` is about the most tokens of one
    sequence and only picks the kernel."""
    pages = _pages(k_pages, v_pages)
    device = k_pages.device
    st = _seqs(device, table, seq_lens, seqs)

    def call(qp, ptr, t, mq, hq, pg, sq, sc, o, code, l, w, wb, s):
        return B.load().attn_paged_fwd(qp, ptr, t, mq, hq, ctypes.byref(pg), ctypes.byref(sq), sc, int(window), int(sinks),
                                       o, code, l, w, wb, s)
    return _attend("attn_paged_fwd", q, pages, st, device, scale, q_ptr, max_q, out, lse, out_dtype, ws, stream, call, 0)


def attn_prefix_fwd(q, k_pages, v_pages, prefix_table, prefix_lens, group_ptr, table, seq_lens, scale: float,
                    q_ptr=None, max_q=None, seqs=None, out=None, lse=None, out_dtype=None, ws=None, stream=None):
    """O, lse of sequences whose groups share a prefix that is read once.

    Sequences group_ptr[g] .. group_ptr[g+1] see the prefix of row g of
    prefix_table / prefix_lens, then their own keys as in ``attn_paged_fwd``
    (seq_lens counts the tokens behind the prefix)."""
    pages = _pages(k_pages, v_pages)
    device = k_pages.device
    st = _seqs(device, table, seq_lens, seqs)
    pre = _seqs(device, prefix_table, prefix_lens, None, "prefix_")
    _ints(device, group_ptr=group_ptr)
    if group_ptr.shape[0] != pre.n_seqs + 1:
        raise ValueError("group_ptr must have one entry a prefix and one more")

    def call(qp, ptr, t, mq, hq, pg, sq, sc, o, code, l, w, wb, s):
        return B.load().attn_prefix_fwd(qp, ptr, t, mq, hq, ctypes.byref(pg), ctypes.byref(pre), group_ptr.data_ptr(),
                                        ctypes.byref(sq), sc, o, code, l, w, wb, s)
    return _attend("attn_prefix_fwd", q, pages, st, device, scale, q_ptr, max_q, out, lse, out_dtype, ws, stream, call, 1)


def attn_cache_extend(table, seq_lens, refs, seqs, counts, page_size: int, stream=None):
    """Adds counts[i] tokens to row seqs[i] of the cache: the lowest free pages
    are taken for them, in the list's order, and the lengths grow."""
    c = _cache(table, seq_lens, refs, page_size)
    _lists(table.device, seqs, counts)
    with _On(table.device):
        B._check(B.load().attn_cache_extend(ctypes.byref(c), seqs.data_ptr(), counts.data_ptr(), seqs.shape[0],
                                            B._stream_ptr(stream)), "attn_cache_extend")


def attn_cache_free(table, seq_lens, refs, seqs, page_size: int, stream=None):
    """Empties the listed rows; pages that nobody else holds become free."""
    c = _cache(table, seq_lens, refs, page_size)
    _lists(table.device, seqs)
    with _On(table.device):
        B._check(B.load().attn_cache_free(ctypes.byref(c), seqs.data_ptr(), seqs.shape[0], B._stream_ptr(stream)),
                 "attn_cache_free")


def attn_cache_trim(table, seq_lens, refs, page_size: int, window: int, sinks: int = 0, seqs=None, stream=None):
    """Gives back the pages (of all rows, or the listed ones) that no token at
    position seq_len - 1 or later sees through the window."""
    c = _cache(table, seq_lens, refs, page_size)
    if seqs is not None:
        _lists(table.device, seqs)
    with _On(table.device):
        B._check(B.load().attn_cache_trim(ctypes.byref(c), None if seqs is None else seqs.data_ptr(),
                                          c.n_slots if seqs is None else seqs.shape[0], int(window), int(sinks),
                                          B._stream_ptr(stream)), "attn_cache_trim")


def _copies(c, device, cap, n, stream):
    import torch
    nb = ctypes.c_size_t(0)
    B._check(B.load().attn_cache_workspace_bytes(ctypes.byref(c), n, ctypes.byref(nb)), "attn_cache_workspace_bytes")
    copies = torch.empty(1 + 2 * cap, dtype=torch.int32, device=device)
    ws = torch.empty(nb.value, dtype=torch.uint8, device=device)
    if stream is not None:
        _borrowed(stream, copies, ws)
    return copies, ws


def attn_cache_fork(table, seq_lens, refs, src, dst, page_size: int, stream=None):
    """Row dst[i] becomes what row src[i] was, for all i at once: full pages are
    shared, partial ones copied.  Returns the copy list for
    ``attn_cache_copy_pages``."""
    c = _cache(table, seq_lens, refs, page_size)
    _lists(table.device, src, dst, ("src", "dst"))
    n = src.shape[0]
    with _On(table.device):
        copies, ws = _copies(c, table.device, n, n, stream)
        B._check(B.load().attn_cache_fork(ctypes.byref(c), src.data_ptr(), dst.data_ptr(), n, copies.data_ptr(), n,
                                          ws.data_ptr(), ws.numel(), B._stream_ptr(stream)), "attn_cache_fork")
    return copies


def attn_cache_compact(table, seq_lens, refs, page_size: int, stream=None):
    """Moves the pages in use to the lowest indices.  Returns the copy list for
    ``attn_cache_copy_pages``."""
    c = _cache(table, seq_lens, refs, page_size)
    cap = c.n_pages // 2
    with _On(table.device):
        copies, ws = _copies(c, table.device, cap, 0, stream)
        B._check(B.load().attn_cache_compact(ctypes.byref(c), copies.data_ptr(), cap, ws.data_ptr(), ws.numel(),
                                             B._stream_ptr(stream)), "attn_cache_compact")
    return copies


def attn_cache_copy_pages(pools, copies, stream=None):
    """Copies whole pages inside every tensor of ``pools`` ([n_pages, ...],
    each page contiguous, alike in size): page copies[1 + i] to page
    copies[1 + cap + i] for i < copies[0], copies int32 [1 + 2 cap]."""
    pools = list(pools)
    if not pools:
        return
    x = pools[0]
    n, page, stride = x.shape[0], x[0].numel() * x.element_size(), x.stride(0) * x.element_size()
    for y in pools:
        if not y.is_cuda or y.device != x.device or y.shape[0] != n or not y[0].is_contiguous() or \
                y[0].numel() * y.element_size() != page or (n > 1 and y.stride(0) * y.element_size() != stride):
            raise ValueError("pools must be tensors [n_pages, ...] on one CUDA device, alike in page size, each page contiguous")
    _ints(x.device, copies=copies)
    if copies.shape[0] % 2 != 1:
        raise ValueError("copies must be int32 [1 + 2 cap]")
    ptrs = (ctypes.c_void_p * len(pools))(*[y.data_ptr() for y in pools])
    with _On(x.device):
        B._check(B.load().attn_cache_copy_pages(ptrs, len(pools), page, max(stride, page) if n == 1 else stride, n,
                                                copies.data_ptr(), copies.shape[0] // 2, B._stream_ptr(stream)),
                 "attn_cache_copy_pages")


def attn_cache_write(k_pages, v_pages, k_new, v_new, table, seq_lens, q_ptr=None, seqs=None, stream=None):
    """Writes the newest tokens' keys and values ([n_tokens,H_k,d] bf16, d
    contiguous) to the ends of their sequences (q_ptr, seqs as in
    ``attn_paged_fwd``; seq_lens counts them already)."""
    import torch
    pages = _pages(k_pages, v_pages)
    device = k_pages.device
    st = _seqs(device, table, seq_lens, seqs)
    _ints(device, q_ptr=q_ptr)
    if q_ptr is not None and q_ptr.shape[0] != st.n_seqs + 1:
        raise ValueError("q_ptr must have one entry a sequence and one more")
    if k_new.dtype != torch.bfloat16 or v_new.dtype != torch.bfloat16 or k_new.device != device or v_new.device != device or \
            k_new.dim() != 3 or k_new.shape[1:] != (pages.hk, pages.d) or k_new.shape != v_new.shape or \
            k_new.stride() != v_new.stride() or k_new.stride(2) != 1:
        raise ValueError("k_new and v_new must be bf16 [n_tokens, H_k, d] on the pages' device, alike in strides, d contiguous")
    with _On(device):
        B._check(B.load().attn_cache_write(ctypes.byref(pages), ctypes.byref(st), None if q_ptr is None else q_ptr.data_ptr(),
                                           k_new.data_ptr(), v_new.data_ptr(), k_new.shape[0], k_new.stride(0), k_new.stride(1),
                                           B._stream_ptr(stream)), "attn_cache_write")


def attn_slices_from_windows(lengths: Sequence[int], window: int, sinks: int = 0) -> np.ndarray:
    """Windowed causal mask of packed sequences -> slice list (host), for
    ``attn_build_tiles``: a token sees its sequence's keys j <= i with
    j > i - window or j < sinks (window 0: all)."""
    a = np.ascontiguousarray(np.asarray(lengths, dtype=np.int32).reshape(-1))
    n = ctypes.c_int(0)
    out = np.zeros((max(1, 3 * len(a)), 5), dtype=np.int32)
    B._check(B.load().attn_slices_from_windows(a.ctypes.data, len(a), int(window), int(sinks), out.ctypes.data,
                                               3 * len(a), ctypes.byref(n)), "attn_slices_from_windows")
    return out[:n.value]


def _declare(lib):
    vp, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    pages, seqs = ctypes.POINTER(AttnPages), ctypes.POINTER(AttnSeqs)
    lib.attn_paged_workspace_bytes.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.attn_paged_fwd.argtypes = [vp, vp, i32, i32, i32, pages, seqs, f32, i32, i32, vp, i32, vp, vp, sz, vp]
    lib.attn_prefix_fwd.argtypes = [vp, vp, i32, i32, i32, pages, seqs, vp, seqs, f32, vp, i32, vp, vp, sz, vp]
    cache = ctypes.POINTER(AttnCache)
    lib.attn_cache_extend.argtypes = [cache, vp, vp, i32, vp]
    lib.attn_cache_free.argtypes = [cache, vp, i32, vp]
    lib.attn_cache_trim.argtypes = [cache, vp, i32, i32, i32, vp]
    lib.attn_cache_workspace_bytes.argtypes = [cache, i32, ctypes.POINTER(sz)]
    lib.attn_cache_fork.argtypes = [cache, vp, vp, i32, vp, i32, vp, sz, vp]
    lib.attn_cache_compact.argtypes = [cache, vp, i32, vp, sz, vp]
    lib.attn_cache_copy_pages.argtypes = [vp, i32, sz, sz, i32, vp, i32, vp]
    lib.attn_cache_write.argtypes = [pages, seqs, vp, vp, vp, i32, ctypes.c_int64, ctypes.c_int64, vp]
    lib.attn_slices_from_windows.argtypes = [vp, i32, i32, i32, vp, i32, ctypes.POINTER(ctypes.c_int)]
