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
    see[:, max(base, 0):] = bits[:, max(-base, 0):]         # drafts before entry 0 are not there
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


# ------------------------------------------------------------------------------ pages
class Pages:
    """Page bookkeeping and data of a cache, one entry and one page at a time.

    pools: list of uint8 arrays [pages, heads, 64, row]; table [B, ld], lens [B], ref [pages],
    free [pages] with n_free of them on the stack.
    """

    def __init__(self, pools, table, lens, ref, free, n_free):
        self.pools, self.table, self.lens = pools, table, lens
        self.ref, self.free, self.n_free = ref, free, n_free

    def copy(self):
        return Pages([p.copy() for p in self.pools], self.table.copy(), self.lens.copy(), self.ref.copy(),
                     self.free.copy(), self.n_free)

    def _good(self, page):
        return 0 <= page < len(self.ref)

    def _push(self, gone):
        for page in sorted(gone):
            self.free[self.n_free] = page
            self.n_free += 1

    def _drop(self, page, gone):
        self.ref[page] -= 1
        if self.ref[page] == 0:
            gone.add(int(page))

    def _pop(self, rank, have):
        return self.free[have - 1 - rank]

    def _first(self, req):
        """Entries whose request is in range and not named by an earlier one."""
        seen, ok = set(), []
        for r in req:
            ok.append(0 <= r < len(self.lens) and r not in seen)
            seen.add(r)
        return ok

    def free_requests(self, req, new=None):
        new = [0] * len(req) if new is None else new
        ok = [f and 0 <= n <= self.lens[r] for f, r, n in zip(self._first(req), req, new)]
        gone = set()
        for r, n, good in zip(req, new, ok):
            if good:
                self._cut(r, n, gone)
        self._push(gone)
        return [int(x) for x in ok]

    def _cut(self, r, n, gone):
        for c in range(-(-n // PAGE), -(-int(self.lens[r]) // PAGE)):
            page = self.table[r, c]
            self.table[r, c] = -1
            if self._good(page):
                self._drop(page, gone)
        self.lens[r] = n

    def fork(self, src, dst, deep):
        lens, have, used, ok, short = self.lens.copy(), self.n_free, 0, [], False
        for f, s, d in zip(self._first(dst), src, dst):
            good = f and 0 <= s < len(lens) and s != d and lens[d] == 0
            if good:
                L = int(lens[s])
                need = -(-L // PAGE) if deep else int(L % PAGE != 0)
                used += need
                good = used <= have
            ok.append(int(good))
            if not good:
                continue
            rank = used - need
            for c in range(-(-L // PAGE)):
                old = self.table[s, c]
                if not deep and c < L // PAGE:
                    self.table[d, c] = old
                    if self._good(old):
                        self.ref[old] += 1
                    continue
                page = self._pop(rank, have)
                rank += 1
                self.table[d, c] = page
                self.ref[page] = 1
                if self._good(old):
                    for p in self.pools:
                        p[page] = p[old]
            self.lens[d] = L
            self.n_free = have - used
        return ok

    def grow(self, req, new):
        have, used, ok, gone = self.n_free, 0, [], set()
        ref = self.ref.copy()                       # sharing is judged as it was before the call
        taken = 0
        for f, r, n in zip(self._first(req), req, new):
            good = f and n >= self.lens[r] and -(-n // PAGE) <= self.table.shape[1]
            if good:
                old = int(self.lens[r])
                c0, c1 = -(-old // PAGE), -(-n // PAGE)
                last = self.table[r, old // PAGE] if old % PAGE and n > old else -1
                cow = self._good(last) and ref[last] > 1
                need = c1 - c0 + int(cow)
                used += need
                good = used <= have
            ok.append(int(good))
            if not good:
                continue
            rank = used - need
            for c in range(c0 - int(cow), c1):
                page = self._pop(rank, have)
                rank += 1
                if cow and c == c0 - 1:
                    for p in self.pools:
                        p[page] = p[last]
                    self._drop(last, gone)
                self.table[r, c] = page
                self.ref[page] = 1
            self.lens[r] = n
            taken = used
        self.n_free = have - taken
        self._push(gone)
        return ok

    def compact(self, req, start, keep, n_keep):
        ok = []
        for i, (f, r) in enumerate(zip(self._first(req), req)):
            ks = [int(x) for x in keep[i][:max(0, n_keep[i])]]
            good = f and 0 <= n_keep[i] <= len(keep[i]) and 0 <= start[i] <= self.lens[r] and \
                all(start[i] <= k < self.lens[r] for k in ks) and all(a < b for a, b in zip(ks, ks[1:]))
            if good:
                for j, k in enumerate(ks):
                    if k != start[i] + j:
                        a, b = self.table[r, k // PAGE], self.table[r, (start[i] + j) // PAGE]
                        good = good and self._good(a) and self._good(b) and self.ref[b] == 1
            ok.append(int(good))
        gone = set()
        for i, r in enumerate(req):
            if not ok[i]:
                continue
            for j, k in enumerate(keep[i][:n_keep[i]]):
                d = start[i] + j
                if k != d:
                    for p in self.pools:
                        p[self.table[r, d // PAGE], :, d % PAGE] = p[self.table[r, k // PAGE], :, k % PAGE]
            self._cut(r, start[i] + n_keep[i], gone)
        self._push(gone)
        return ok


# ------------------------------------------------------------------------------ norms and rotation
def qk_norm_rope(x, weight, eps, pos, inv_freq, first, halves):
    """x [T, heads, D] (float64) normed (weight None: not) and rotated; pos [T]."""
    x = np.array(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    n = len(inv_freq)
    a, b = (first + np.arange(n), first + n + np.arange(n)) if halves else \
        (first + 2 * np.arange(n), first + 2 * np.arange(n) + 1)
    ang = np.asarray(pos, np.float64)[:, None, None] * np.asarray(inv_freq)[None, None]
    u, v = x[..., a], x[..., b]
    out = x.copy()
    out[..., a] = u * np.cos(ang) - v * np.sin(ang)
    out[..., b] = u * np.sin(ang) + v * np.cos(ang)
    return out
