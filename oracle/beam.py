"""A beam search's choice in float64 from the definition: all continuations of a
prompt, sorted by score and then by place.  Shares no code with the CUDA path.
Pinned by ``tests/test_oracle_beam.py``."""
import numpy as np


def oracle_beam_select(logits, scores, done=None, eos=-1, keep=None):
    """logits [G * B, V], scores [G, B] -> scores, parents, tokens, done, each
    [G, keep] (scores float64), and the sorted scores of all continuations, from
    which ties and gaps are seen."""
    scores = np.asarray(scores, np.float64)
    G, B = scores.shape
    V = logits.shape[1]
    keep = B if keep is None else keep
    x = np.asarray(logits, np.float64).reshape(G, B, V)
    out = np.empty((G, keep)), np.empty((G, keep), int), np.empty((G, keep), int), np.empty((G, keep), bool)
    ranked = np.empty((G, B * V))
    for g in range(G):
        c = np.full((B, V), -np.inf)
        for b in range(B):
            s = scores[g, b]
            if not np.isfinite(s):
                continue
            if done is not None and done[g, b]:
                c[b, eos] = s
                continue
            row = x[g, b]
            if np.isnan(row).any() or np.isposinf(row).any() or np.isneginf(row).all():
                continue
            top = row.max()
            c[b] = s + (row - (top + np.log(np.exp(row - top).sum())))
        flat = c.ravel()
        order = np.lexsort((np.arange(flat.size), -flat))
        ranked[g] = flat[order]
        best = order[:keep]
        out[0][g], out[1][g], out[2][g] = flat[best], g * B + best // V, best % V
        for i, j in enumerate(best):
            out[3][g, i] = (done is not None and bool(done[g, j // V])) or j % V == eos
    return out + (ranked,)
