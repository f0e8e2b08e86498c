"""GB300 (sm_103a) masked-attention forward behind a small C ABI.

    tiles      = attn_build_tiles(slices, S_q, S_k)        # slice list -> CSR tile metadata
    out, lse   = attn_fwd(q, k, v, tiles, scale)           # softmax(scale QK^T + mask) V, row LSE
    out, lse   = attn_merge([o_1, o_2, ...], [lse_1, ...]) # exact KV-split merge

    out, lse   = attn_paged_fwd(q, k_pages, v_pages, table, seq_lens, scale, ...)   # over a paged cache
    out, lse   = attn_prefix_fwd(...)                      # groups that share a prefix
    attn_cache_extend / write / read / fork / free / trim / compact / copy_pages    # that cache's pages
    scores, parents, tokens, done = attn_beam_select(logits, scores, ...)           # a beam search's step
    attn_beam_reorder(states, parents)

All run as hand-written CUDA kernels in ``libattn_slice.so`` (see
``include/attn_slice.h``, ``attn_paged.h`` and ``attn_beam.h``); this package only
marshals arguments.
"""
from .beam import attn_beam_reorder, attn_beam_select
from .binding import (ATTN_DTYPE_BF16, ATTN_DTYPE_F32, ATTN_FWD_TILE_K, ATTN_FWD_TILE_Q,
                      AttnError, Tiles, attn_build_tiles, attn_bwd, attn_fwd, attn_last_device_error,
                      attn_merge, attn_selftest_wait_timeout, attn_set_exp2_poly,
                      attn_set_wait_limit_ns, attn_slices_from_block_grid,
                      attn_tiles_workspace_bytes, load)
from .paging import (attn_cache_compact, attn_cache_copy_pages, attn_cache_extend, attn_cache_fork,
                     attn_cache_free, attn_cache_read, attn_cache_trim, attn_cache_write,
                     attn_paged_fwd, attn_prefix_fwd, attn_slices_from_windows)

__all__ = ["attn_build_tiles", "attn_fwd", "attn_bwd", "attn_merge", "attn_slices_from_block_grid",
           "attn_tiles_workspace_bytes", "attn_last_device_error", "attn_set_wait_limit_ns",
           "attn_set_exp2_poly",
           "attn_selftest_wait_timeout", "Tiles", "AttnError", "load",
           "attn_paged_fwd", "attn_prefix_fwd", "attn_slices_from_windows",
           "attn_cache_extend", "attn_cache_write", "attn_cache_fork", "attn_cache_free", "attn_cache_trim",
           "attn_cache_compact", "attn_cache_copy_pages", "attn_cache_read",
           "attn_beam_select", "attn_beam_reorder",
           "ATTN_DTYPE_BF16", "ATTN_DTYPE_F32", "ATTN_FWD_TILE_Q", "ATTN_FWD_TILE_K"]
