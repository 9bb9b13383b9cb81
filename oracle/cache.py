"""Plain fp64 forms of the paged-cache operators (test infrastructure, like the rest of oracle/).

A cache here is numpy arrays: pools [pages, kv heads, 64, row], a block table [B, ld] and lengths.
Nothing is shared with the HIP sources; every function follows the definitions in include/fm.h
one entry at a time where that is affordable.
"""
from __future__ import annotations

import numpy as np

PAGE = 64


def entry(table_row, s, n_phys):
    """(page, slot) of entry s, or None where its page is not mapped."""
    page = int(table_row[s // PAGE])
    return (page, s % PAGE) if 0 <= page < n_phys else None


def window_rows(n: int, length: int, window: int, n_sink: int) -> np.ndarray:
    """Visible entries [n, length] of the last n entries' rows."""
    pos = np.arange(length - n, length)[:, None]
    s = np.arange(length)[None]
    return (s <= pos) & ((s > pos - window) | (s < n_sink))


def tree_rows(bits: np.ndarray, length: int, window: int, n_sink: int) -> np.ndarray:
    """Visible entries [n, length] of n drafts; bits [n, n]: row i sees draft j."""
    n = bits.shape[0]
    base = length - n
    pos = base + bits.sum(1)[:, None].astype(np.int64) - 1
    s = np.arange(length)[None]
    see = (s < base) & (s <= pos) & ((s > pos - window) | (s < n_sink))
    see[:, base:] = bits
    return see


def attend(q, k, v, see, scale):
    """One request: q [n, H, D], k and v [L, K, D] (float64), see [n, L].

    Returns out [n, H, D], lse [n, H], and for tolerances: sum p |v| [n, H, D], the largest
    scale sum |q k| of a row's visible entries [n, H], and the visible entries of a row [n].
    Hidden entries take no part at all, whatever they hold.
    """
    n, H, D = q.shape
    G = H // k.shape[1]
    out, mag = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, big = np.full((n, H), -np.inf), np.zeros((n, H))
    for i in range(n):
        at = np.flatnonzero(see[i])
        if not len(at):
            continue
        for h in range(H):
            kk, vv = k[at, h // G], v[at, h // G]
            with np.errstate(invalid="ignore", over="ignore"):
                x = scale * (kk * q[i, h]).sum(1)
                big[i, h] = scale * np.max(np.abs(kk) @ np.abs(q[i, h]))
                m = x.max()
                if m == -np.inf:
                    continue
                e = np.exp(x - m)
                out[i, h] = (e[:, None] * vv).sum(0) / e.sum()
                mag[i, h] = (e[:, None] * np.abs(vv)).sum(0) / e.sum()
                lse[i, h] = m + np.log(e.sum())
    return out, lse, mag, big, see.sum(1)
