"""Python entry points of ``include/attn_beam.h``: a beam search's step over the
sequences of a paged cache.

Argument marshalling only, in ``csrc/paging_module.cpp``, as in ``paging``.  A
call runs on its tensors' device, on ``stream`` or that device's current stream.
"""
from __future__ import annotations

import ctypes

from . import paging as P


def attn_beam_select(logits, scores, done=None, eos: int = -1, slots=None, keep=None, ws=None, stream=None):
    """The ``keep`` (None: beams) best continuations of every prompt.

    logits [groups * beams, vocab] f32 or bf16; scores f32 [groups, beams];
    done bool or uint8 [groups, beams] (ended beams go on as they are, by the
    token ``eos``).  Returns scores, parents, tokens, done, all [groups, keep],
    best first: score[b] + logit - ln sum exp(logits of b), the parent's row
    g * beams + b, the token, and whether the beam has ended.  Equal ones stand in
    the order of beam, then token.  With ``slots`` (int32 [groups * beams], each
    beam's row of the page table) a fifth: slots[parents], the ``src`` of
    ``attn_cache_fork``.  A ``stream`` other than the current one waits for what
    the current one holds; what follows on the current one does not wait for it."""
    made = ()
    if stream is not None:
        import torch
        here = torch.cuda.current_stream(logits.device)
        if stream != here:
            # outputs and workspace are then made on that stream, and it waits for what they follow
            stream.wait_stream(here)
            with torch.cuda.stream(stream):
                made = P._m().beam_select(logits, scores, done, eos, slots, keep, ws, stream.cuda_stream)
            for x in made:
                x.record_stream(here)
            return made
        stream = stream.cuda_stream
    return (P._module or P._m()).beam_select(logits, scores, done, eos, slots, keep, ws, stream)


def attn_beam_reorder(states, parents, stream=None):
    """Row i of every tensor of ``states`` ([groups * beams, ...], each row
    contiguous) becomes what row parents[i] was, in place; parents int32
    [groups, beams], each within its own group.  A ``stream`` other than the
    current one waits for what the current one holds, as in ``attn_beam_select``."""
    if stream is not None:
        import torch
        here = torch.cuda.current_stream(parents.device)
        if stream != here:
            stream.wait_stream(here)
        stream = stream.cuda_stream
    (P._module or P._m()).beam_reorder(states, parents, stream)


def _declare(lib):
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.attn_beam_workspace_bytes.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.attn_beam_select.argtypes = [vp, i32, i64, i32, i32, i32, vp, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.attn_beam_reorder.argtypes = [vp, vp, vp, i32, vp, i32, i32, vp]
