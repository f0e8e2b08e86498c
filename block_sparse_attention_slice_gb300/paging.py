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
import functools
import struct
from typing import Sequence

import numpy as np
import torch

from . import binding as B

# The C structs, packed in one step: a call of a few microseconds on the GPU
# is not to wait for field-by-field marshalling.
_PAGES = struct.Struct("@PPiiiiqqq").pack      # attn_pages_t
_SEQS = struct.Struct("@PPPqiiii").pack        # attn_seqs_t
_CACHE = struct.Struct("@PPPqiiii").pack       # attn_cache_t
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _ints(device, name, x):
    """Address of an int32 vector on `device`, contiguous; None stays None."""
    if x is None:
        return None
    if x.dtype is not _I32 or x.dim() != 1 or x.device != device or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 vector on {device}")
    return x.data_ptr()


def _pages(k, v):
    """attn_pages_t, the device, H_k and d."""
    st = k.stride()
    if k.dim() != 4 or k.shape != v.shape or st != v.stride() or st[3] != 1:
        raise ValueError("k_pages and v_pages must be [n_pages, page_size, H_k, d], alike in strides, d contiguous")
    device = k.device
    if k.dtype is not _BF16 or v.dtype is not _BF16 or not k.is_cuda or v.device != device:
        raise ValueError("k_pages and v_pages must be bf16 tensors on one CUDA device")
    n, page, hk, d = k.shape
    return _PAGES(k.data_ptr(), v.data_ptr(), n, page, hk, d, st[0], st[1], st[2]), device, hk, d


def _rows(device, table, seq_lens, what=""):
    """Checks a table with its lengths: address, lengths' address, row stride, slots, columns."""
    if table.dtype is not _I32 or table.dim() != 2 or table.device != device:
        raise ValueError(f"{what}table must be int32 [n_slots, max_pages] on {device}")
    n, width = table.shape
    stride, inner = table.stride()
    if inner != 1 and width > 1:
        raise ValueError(f"{what}table must have contiguous rows")
    lens = _ints(device, what + "seq_lens", seq_lens)
    if seq_lens.shape[0] != n:
        raise ValueError(f"{what}table and {what}seq_lens must have one row a slot")
    return table.data_ptr(), lens, stride if n > 1 else max(width, stride), n, width


def _seqs(device, table, seq_lens, seqs, what=""):
    """attn_seqs_t and the number of sequences."""
    at, lens, stride, n, width = _rows(device, table, seq_lens, what)
    if seqs is None:
        return _SEQS(at, lens, 0, stride, n, width, n, 0), n
    m = seqs.shape[0]
    return _SEQS(at, lens, _ints(device, "seqs", seqs), stride, n, width, m, 0), m


def _cache(table, seq_lens, refs, page_size):
    """attn_cache_t and the device."""
    device = table.device
    if not table.is_cuda:
        raise ValueError("the cache's arrays must be CUDA tensors")
    at, lens, stride, n, width = _rows(device, table, seq_lens)
    return _CACHE(at, lens, _ints(device, "refs", refs), stride, n, width, refs.shape[0], int(page_size)), device


def _call(device, stream, name, *args):
    """The C entry `name` on the tensors' device, on `stream` or that device's current one."""
    s = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream
    fn = getattr(B.load(), name)
    if torch.cuda.current_device() == device.index:
        code = fn(*args, s)
    else:
        with torch.cuda.device(device):
            code = fn(*args, s)
    if code:
        raise B.AttnError(code, name)


def _borrowed(stream, *tensors):
    """Tensors allocated here on the current stream and used on another one."""
    if stream is not None:
        here = torch.cuda.current_stream(tensors[0].device)
        if stream != here:
            stream.wait_stream(here)
            for x in tensors:
                x.record_stream(stream)


@functools.lru_cache(maxsize=1024)
def _workspace(index, t, hq, d, prefix):
    """Bytes of workspace of a call of these sizes on device `index`."""
    nb = ctypes.c_size_t(0)
    with torch.cuda.device(index):
        B._check(B.load().attn_paged_workspace_bytes(t, hq, d, prefix, ctypes.byref(nb)), "attn_paged_workspace_bytes")
    return nb.value


def _attend(q, device, hk, d, q_ptr, n_seqs, max_q, out, lse, out_dtype, ws, stream, prefix):
    """Checks and outputs that both attention calls share: the C arguments before and behind their own."""
    if q.dtype is not _BF16 or q.dim() != 3 or q.device != device or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous bf16 [n_tokens, H, d] tensor on {device}")
    t, hq, dq = q.shape
    if dq != d:
        raise ValueError("q and the pages must have one head dim")
    ptr = _ints(device, "q_ptr", q_ptr)
    if q_ptr is not None and q_ptr.shape[0] != n_seqs + 1:
        raise ValueError("q_ptr must have one entry a sequence and one more")
    made = []
    if out is None:
        out = torch.empty_like(q, dtype=out_dtype)
        made.append(out)
    elif out.shape != q.shape or out.device != device or not out.is_contiguous() or out_dtype not in (None, out.dtype):
        raise ValueError("out must be a contiguous bf16 or f32 tensor like q")
    if out.dtype is not _BF16 and out.dtype is not _F32:
        raise ValueError("out must be bf16 or f32")
    if lse is None:
        lse = torch.empty((hq, t), dtype=_F32, device=device)
        made.append(lse)
    elif lse.shape != (hq, t) or lse.dtype is not _F32 or lse.device != device or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous f32 [H, n_tokens] tensor")
    if ws is None:
        ws = torch.empty(_workspace(device.index, t, hq, d, prefix), dtype=torch.uint8, device=device)
        made.append(ws)
    elif ws.device != device or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous tensor on the queries' device")
    if stream is not None and made:
        _borrowed(stream, *made)
    if max_q is None:
        max_q = 1 if q_ptr is None else max(1, t)
    code = B.ATTN_DTYPE_F32 if out.dtype is _F32 else B.ATTN_DTYPE_BF16
    return out, lse, (q.data_ptr(), ptr, t, int(max_q), hq), (out.data_ptr(), code, lse.data_ptr(), ws.data_ptr(),
                                                              ws.numel() * ws.element_size())


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
    pages, device, hk, d = _pages(k_pages, v_pages)
    rows, n = _seqs(device, table, seq_lens, seqs)
    out, lse, before, behind = _attend(q, device, hk, d, q_ptr, n, max_q, out, lse, out_dtype, ws, stream, 0)
    _call(device, stream, "attn_paged_fwd", *before, pages, rows, scale, window, sinks, *behind)
    return out, lse


def attn_prefix_fwd(q, k_pages, v_pages, prefix_table, prefix_lens, group_ptr, table, seq_lens, scale: float,
                    q_ptr=None, max_q=None, seqs=None, out=None, lse=None, out_dtype=None, ws=None, stream=None):
    """O, lse of sequences whose groups share a prefix that is read once.

    Sequences group_ptr[g] .. group_ptr[g+1] see the prefix of row g of
    prefix_table / prefix_lens, then their own keys as in ``attn_paged_fwd``
    (seq_lens counts the tokens behind the prefix)."""
    pages, device, hk, d = _pages(k_pages, v_pages)
    rows, n = _seqs(device, table, seq_lens, seqs)
    pre, groups = _seqs(device, prefix_table, prefix_lens, None, "prefix_")
    first = _ints(device, "group_ptr", group_ptr)
    if group_ptr.shape[0] != groups + 1:
        raise ValueError("group_ptr must have one entry a prefix and one more")
    out, lse, before, behind = _attend(q, device, hk, d, q_ptr, n, max_q, out, lse, out_dtype, ws, stream, 1)
    _call(device, stream, "attn_prefix_fwd", *before, pages, pre, first, rows, scale, *behind)
    return out, lse


def attn_cache_extend(table, seq_lens, refs, seqs, counts, page_size: int, stream=None):
    """Adds counts[i] tokens to row seqs[i] of the cache: the lowest free pages
    are taken for them, in the list's order, and the lengths grow."""
    c, device = _cache(table, seq_lens, refs, page_size)
    if counts.shape != seqs.shape:
        raise ValueError("seqs and counts must be of one length")
    _call(device, stream, "attn_cache_extend", c, _ints(device, "seqs", seqs), _ints(device, "counts", counts), seqs.shape[0])


def attn_cache_free(table, seq_lens, refs, seqs, page_size: int, stream=None):
    """Empties the listed rows; pages that nobody else holds become free."""
    c, device = _cache(table, seq_lens, refs, page_size)
    _call(device, stream, "attn_cache_free", c, _ints(device, "seqs", seqs), seqs.shape[0])


def attn_cache_trim(table, seq_lens, refs, page_size: int, window: int, sinks: int = 0, seqs=None, stream=None):
    """Gives back the pages (of all rows, or the listed ones) that no token at
    position seq_len - 1 or later sees through the window."""
    c, device = _cache(table, seq_lens, refs, page_size)
    _call(device, stream, "attn_cache_trim", c, _ints(device, "seqs", seqs), table.shape[0] if seqs is None else seqs.shape[0],
          window, sinks)


def _copies(device, c, cap, n, stream):
    nb = ctypes.c_size_t(0)
    B._check(B.load().attn_cache_workspace_bytes(c, n, ctypes.byref(nb)), "attn_cache_workspace_bytes")
    copies = torch.empty(1 + 2 * cap, dtype=_I32, device=device)
    ws = torch.empty(nb.value, dtype=torch.uint8, device=device)
    if stream is not None:
        _borrowed(stream, copies, ws)
    return copies, (copies.data_ptr(), cap, ws.data_ptr(), nb.value)


def attn_cache_fork(table, seq_lens, refs, src, dst, page_size: int, stream=None):
    """Row dst[i] becomes what row src[i] was, for all i at once: full pages are
    shared, partial ones copied.  Returns the copy list for
    ``attn_cache_copy_pages``."""
    c, device = _cache(table, seq_lens, refs, page_size)
    if src.shape != dst.shape:
        raise ValueError("src and dst must be of one length")
    n = src.shape[0]
    a, b = _ints(device, "src", src), _ints(device, "dst", dst)
    copies, rest = _copies(device, c, n, n, stream)
    _call(device, stream, "attn_cache_fork", c, a, b, n, *rest)
    return copies


def attn_cache_compact(table, seq_lens, refs, page_size: int, stream=None):
    """Moves the pages in use to the lowest indices.  Returns the copy list for
    ``attn_cache_copy_pages``."""
    c, device = _cache(table, seq_lens, refs, page_size)
    copies, rest = _copies(device, c, refs.shape[0] // 2, 0, stream)
    _call(device, stream, "attn_cache_compact", c, *rest)
    return copies


def attn_cache_copy_pages(pools, copies, stream=None):
    """Copies whole pages inside every tensor of ``pools`` ([n_pages, ...],
    each page contiguous, alike in size): page copies[1 + i] to page
    copies[1 + cap + i] for i < copies[0], copies int32 [1 + 2 cap]."""
    if not pools:
        return
    x = pools[0]
    device, shape, strides, size = x.device, x.shape, x.stride(), x.element_size()
    if not x.is_cuda or x.dim() < 2 or not x[0].is_contiguous():
        raise ValueError("pools must be CUDA tensors [n_pages, ...], each page contiguous")
    n, page = shape[0], shape[1:].numel() * size
    ptrs = []
    for y in pools:
        if y.shape != shape or y.stride() != strides or y.element_size() != size or y.device != device:
            raise ValueError("pools must be alike in shape, strides and element size, on one device")
        ptrs.append(y.data_ptr())
    at = _ints(device, "copies", copies)
    if copies.shape[0] % 2 != 1:
        raise ValueError("copies must be int32 [1 + 2 cap]")
    _call(device, stream, "attn_cache_copy_pages", struct.pack(f"@{len(ptrs)}P", *ptrs), len(ptrs), page,
          strides[0] * size if n > 1 else page, n, at, copies.shape[0] // 2)


def attn_cache_write(k_pages, v_pages, k_new, v_new, table, seq_lens, q_ptr=None, seqs=None, stream=None):
    """Writes the newest tokens' keys and values ([n_tokens,H_k,d] bf16, d
    contiguous) to the ends of their sequences (q_ptr, seqs as in
    ``attn_paged_fwd``; seq_lens counts them already)."""
    pages, device, hk, d = _pages(k_pages, v_pages)
    rows, n = _seqs(device, table, seq_lens, seqs)
    ptr = _ints(device, "q_ptr", q_ptr)
    if q_ptr is not None and q_ptr.shape[0] != n + 1:
        raise ValueError("q_ptr must have one entry a sequence and one more")
    st = k_new.stride()
    if k_new.dtype is not _BF16 or v_new.dtype is not _BF16 or k_new.device != device or v_new.device != device or \
            k_new.dim() != 3 or k_new.shape != v_new.shape or k_new.shape[1:] != (hk, d) or st != v_new.stride() or st[2] != 1:
        raise ValueError("k_new and v_new must be bf16 [n_tokens, H_k, d] on the pages' device, alike in strides, d contiguous")
    _call(device, stream, "attn_cache_write", pages, rows, ptr, k_new.data_ptr(), v_new.data_ptr(), k_new.shape[0], st[0], st[1])


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
    vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    lib.attn_paged_workspace_bytes.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.attn_paged_fwd.argtypes = [vp, vp, i32, i32, i32, vp, vp, f32, i32, i32, vp, i32, vp, vp, sz, vp]
    lib.attn_prefix_fwd.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp, f32, vp, i32, vp, vp, sz, vp]
    lib.attn_cache_extend.argtypes = [vp, vp, vp, i32, vp]
    lib.attn_cache_free.argtypes = [vp, vp, i32, vp]
    lib.attn_cache_trim.argtypes = [vp, vp, i32, i32, i32, vp]
    lib.attn_cache_workspace_bytes.argtypes = [vp, i32, ctypes.POINTER(sz)]
    lib.attn_cache_fork.argtypes = [vp, vp, vp, i32, vp, i32, vp, sz, vp]
    lib.attn_cache_compact.argtypes = [vp, vp, i32, vp, sz, vp]
    lib.attn_cache_copy_pages.argtypes = [vp, i32, sz, sz, i32, vp, i32, vp]
    lib.attn_cache_write.argtypes = [vp, vp, vp, vp, vp, i32, i64, i64, vp]
    lib.attn_slices_from_windows.argtypes = [vp, i32, i32, i32, vp, i32, ctypes.POINTER(ctypes.c_int)]
