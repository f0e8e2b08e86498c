"""Python entry points of ``include/attn_paged.h``: attention over a paged
key/value cache and the pages of that cache.

Argument marshalling only, in ``csrc/paging_module.cpp`` (built beside the CUDA
library as ``_paging``); the computation runs in the CUDA kernels of
``libattn_slice.so``, and there is no fallback.  Index arrays (tables, lengths,
lists) are int32 CUDA tensors and are checked by the kernels; what they find is
reported by ``attn_last_device_error``.

A call runs on its tensors' device, on ``stream`` or that device's current
stream.
"""
from __future__ import annotations

import ctypes
from typing import Sequence

import numpy as np

from . import binding as B

_module = None


def _m():
    """The marshalling module (built by ``__graft_entry__.build()``)."""
    global _module
    if _module is None:
        import torch  # noqa: F401 -- the module's libraries are PyTorch's
        B.load()
        try:
            from . import _paging
        except ImportError as e:
            raise RuntimeError(f"marshalling module not built: run __graft_entry__.build() ({e})") from e
        _paging.set_error(B.AttnError)
        _module = _paging
    return _module


def _on(stream, *tensors):
    """The raw handle of `stream`; tensors allocated on the current stream become its too."""
    import torch
    here = torch.cuda.current_stream(tensors[0].device)
    if stream != here:
        stream.wait_stream(here)
        for x in tensors:
            x.record_stream(stream)
    return stream.cuda_stream


def _made(q, out, lse, out_dtype, ws, d, prefix, stream):
    """Outputs and workspace for a call on another stream than the current one."""
    import torch
    t, hq = q.shape[0], q.shape[1]
    made = []
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype or torch.bfloat16, device=q.device)
        made.append(out)
    if lse is None:
        lse = torch.empty((hq, t), dtype=torch.float32, device=q.device)
        made.append(lse)
    if ws is None:
        nb = ctypes.c_size_t(0)
        with torch.cuda.device(q.device):
            B._check(B.load().attn_paged_workspace_bytes(t, hq, d, prefix, ctypes.byref(nb)), "attn_paged_workspace_bytes")
        ws = torch.empty(nb.value, dtype=torch.uint8, device=q.device)
        made.append(ws)
    return out, lse, ws, _on(stream, *made) if made else stream.cuda_stream


def attn_paged_fwd(q, k_pages, v_pages, table, seq_lens, scale: float, q_ptr=None, max_q=None, window: int = 0,
                   sinks: int = 0, seqs=None, out=None, lse=None, out_dtype=None, ws=None, stream=None):
    """O, lse of each sequence's newest tokens over its cached keys.

    q [n_tokens,H,d] bf16; k_pages/v_pages [n_pages,page_size,H_k,d] bf16;
    table int32 [n_slots,max_pages]; seq_lens int32 [n_slots] (the new tokens,
    whose keys are cached already, included); q_ptr int32 [n_seqs+1] (None:
    one token a sequence); seqs int32 [n_seqs] table rows (None: all, in
    order).  A token at position i sees keys j <= i with j > i - window or
    j < sinks (window 0: all).  ``max_q`` is about the most tokens of one
    sequence and only picks the kernel.  None: 1 without q_ptr, n_tokens with
    it, so give it for batches of short sequences, which otherwise run on the
    kernel of long ones."""
    if stream is not None:
        out, lse, ws, stream = _made(q, out, lse, out_dtype, ws, k_pages.shape[-1], 0, stream)
    return (_module or _m()).paged_fwd(q, k_pages, v_pages, table, seq_lens, scale, q_ptr, max_q, window, sinks, seqs, out, lse,
                                       out_dtype, ws, stream)


def attn_prefix_fwd(q, k_pages, v_pages, prefix_table, prefix_lens, group_ptr, table, seq_lens, scale: float,
                    q_ptr=None, max_q=None, seqs=None, out=None, lse=None, out_dtype=None, ws=None, stream=None):
    """O, lse of sequences whose groups share a prefix that is read once.

    Sequences group_ptr[g] .. group_ptr[g+1] see the prefix of row g of
    prefix_table / prefix_lens, then their own keys as in ``attn_paged_fwd``
    (seq_lens counts the tokens behind the prefix)."""
    if stream is not None:
        out, lse, ws, stream = _made(q, out, lse, out_dtype, ws, k_pages.shape[-1], 1, stream)
    return (_module or _m()).prefix_fwd(q, k_pages, v_pages, prefix_table, prefix_lens, group_ptr, table, seq_lens, scale, q_ptr,
                                        max_q, seqs, out, lse, out_dtype, ws, stream)


def attn_cache_extend(table, seq_lens, refs, seqs, counts, page_size: int, stream=None):
    """Adds counts[i] tokens to row seqs[i] of the cache: the lowest free pages
    are taken for them, in the list's order, and the lengths grow."""
    (_module or _m()).cache_extend(table, seq_lens, refs, seqs, counts, page_size, stream and stream.cuda_stream)


def attn_cache_free(table, seq_lens, refs, seqs, page_size: int, stream=None):
    """Empties the listed rows; pages that nobody else holds become free."""
    (_module or _m()).cache_free(table, seq_lens, refs, seqs, page_size, stream and stream.cuda_stream)


def attn_cache_trim(table, seq_lens, refs, page_size: int, window: int, sinks: int = 0, seqs=None, stream=None):
    """Gives back the pages (of all rows, or the listed ones) that no token at
    position seq_len - 1 or later sees through the window."""
    (_module or _m()).cache_trim(table, seq_lens, refs, page_size, window, sinks, seqs, stream and stream.cuda_stream)


def _list_on(stream, table, cap, bytes_):
    """Copy list and workspace for a call on another stream than the current one."""
    import torch
    copies = torch.empty(1 + 2 * cap, dtype=torch.int32, device=table.device)
    ws = torch.empty(bytes_, dtype=torch.uint8, device=table.device)
    return copies, ws, _on(stream, copies, ws)


def attn_cache_fork(table, seq_lens, refs, src, dst, page_size: int, stream=None):
    """Row dst[i] becomes what row src[i] was, for all i at once: full pages are
    shared, partial ones copied.  Returns the copy list for
    ``attn_cache_copy_pages``."""
    copies = ws = None
    if stream is not None:
        n = src.shape[0]
        copies, ws, stream = _list_on(stream, table, n, max(4 * n * (table.shape[1] + 1), 4 * refs.shape[0]))
    return (_module or _m()).cache_fork(table, seq_lens, refs, src, dst, page_size, copies, ws, stream)


def attn_cache_compact(table, seq_lens, refs, page_size: int, stream=None):
    """Moves the pages in use to the lowest indices.  Returns the copy list for
    ``attn_cache_copy_pages``."""
    copies = ws = None
    if stream is not None:
        copies, ws, stream = _list_on(stream, table, refs.shape[0] // 2, 4 * refs.shape[0])
    return (_module or _m()).cache_compact(table, seq_lens, refs, page_size, copies, ws, stream)


def attn_cache_copy_pages(pools, copies, stream=None):
    """Copies whole pages inside every tensor of ``pools`` ([n_pages, ...],
    each page contiguous, alike in size): page copies[1 + i] to page
    copies[1 + cap + i] for i < copies[0], copies int32 [1 + 2 cap]."""
    (_module or _m()).cache_copy_pages(pools, copies, stream and stream.cuda_stream)


def attn_cache_write(k_pages, v_pages, k_new, v_new, table, seq_lens, q_ptr=None, seqs=None, stream=None):
    """Writes the newest tokens' keys and values ([n_tokens,H_k,d] bf16, d
    contiguous) to the ends of their sequences (q_ptr, seqs as in
    ``attn_paged_fwd``; seq_lens counts them already)."""
    (_module or _m()).cache_write(k_pages, v_pages, k_new, v_new, table, seq_lens, q_ptr, seqs, stream and stream.cuda_stream)


def _int32(x, name):
    """x as int32, refused where that would change a value."""
    a = np.asarray(x)
    with np.errstate(invalid="ignore"):
        b = a.astype(np.int32, order="C")
    if not np.array_equal(a, b):
        raise ValueError(f"{name}: whole numbers of 32 bits are needed")
    return b


def attn_slices_from_windows(lengths: Sequence[int], window: int, sinks: int = 0) -> np.ndarray:
    """Windowed causal mask of packed sequences -> slice list (host), for
    ``attn_build_tiles``: a token sees its sequence's keys j <= i with
    j > i - window or j < sinks (window 0: all)."""
    a = _int32(lengths, "lengths").reshape(-1)
    n = ctypes.c_int(0)
    out = np.zeros((max(1, 3 * len(a)), 5), dtype=np.int32)
    B._check(B.load().attn_slices_from_windows(a.ctypes.data, len(a), int(_int32(window, "window")), int(_int32(sinks, "sinks")),
                                               out.ctypes.data, 3 * len(a), ctypes.byref(n)), "attn_slices_from_windows")
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
