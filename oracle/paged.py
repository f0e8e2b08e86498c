"""Attention over a paged cache in float64, sequence by sequence, from the
definition: a token at position i of its sequence sees the keys j <= i with
j > i - window or j < sinks (window 0: all of them), behind the whole prefix
of its group where there is one.  Shares no code with the CUDA path."""
import numpy as np


def cached_rows(pages, row, n):
    """The first n cached rows [n, H_k, d] of a sequence's table row."""
    j = np.arange(n)
    return pages[row[j // pages.shape[1]], j % pages.shape[1]]


def oracle_paged(q, k_pages, v_pages, table, seq_lens, q_ptr, scale, window=0, sinks=0, seqs=None, prefix=None):
    """q [T,H,d], pages [n_pages,page,H_k,d] float64 arrays; prefix: (table,
    lens, group_ptr) or None.  Returns O, lse [H,T], A and B: O and lse, the
    weighted sum of |v| and the largest scale * sum |q||k| each row met, from
    which rounding bounds are formed.  Rows of no sequence stay NaN."""
    T, H, d = q.shape
    hk = k_pages.shape[2]
    O, A = np.full((T, H, d), np.nan), np.zeros((T, H, d))
    lse, big = np.full((H, T), np.nan), np.zeros((H, T))
    for b in range(len(q_ptr) - 1):
        slot = b if seqs is None else int(seqs[b])
        n, new = int(seq_lens[slot]), int(q_ptr[b + 1] - q_ptr[b])
        k, v = (cached_rows(x, table[slot], n) for x in (k_pages, v_pages))
        m = 0
        if prefix is not None:
            ptable, plens, group_ptr = prefix
            for g in range(len(plens)):
                if group_ptr[g] <= b < group_ptr[g + 1]:
                    m = int(plens[g])
                    k, v = (np.concatenate([cached_rows(x, ptable[g], m), y])
                            for x, y in ((k_pages, k), (v_pages, v)))
        if new == 0:
            continue
        i = np.arange(n - new, n)[:, None]
        j = np.arange(n)[None]
        own = (j <= i) & ((j > i - window) | (j < sinks)) if window else j <= i
        seen = np.concatenate([np.ones((new, m), bool), own], 1)
        some = seen.any(1)
        rows = slice(int(q_ptr[b]), int(q_ptr[b + 1]))
        O[rows], lse[:, rows] = 0.0, -np.inf
        if not some.any():
            continue
        used = seen.any(0)                    # what no row sees takes no part, whatever it is
        seen, kk, vv = seen[some][:, used], k[used], v[used]
        for h in range(H):
            g = h // (H // hk)
            qq = q[rows][some, h]
            s = np.where(seen, qq @ kk[:, g].T * scale, -np.inf)
            top = s.max(1, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(1, keepdims=True)
            O[rows][some, h] = p @ vv[:, g] / total
            A[rows][some, h] = p @ np.abs(vv[:, g]) / total
            lse[h, rows][some] = (top + np.log(total))[:, 0]
            big[h, rows][some] = np.where(seen, np.abs(qq) @ np.abs(kk[:, g]).T, 0.0).max(1) * scale
    return O, lse, A, big
