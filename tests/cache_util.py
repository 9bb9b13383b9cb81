"""Shared pieces of the paged-cache tests: seeded caches, and running the entry points on them."""
from __future__ import annotations

import numpy as np
import torch

from oracle import cache as OC
from top_selection_fm_amd import api

PAGE = 64
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8x132": torch.bfloat16}


def pack_fp8(x: torch.Tensor) -> torch.Tensor:
    """132-byte rows of x [..., 128]."""
    a = x.abs().amax(-1, keepdim=True)
    scale = torch.where(a > 0, a / 448, torch.ones_like(a)).float()
    codes = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.cat([codes, scale.contiguous().view(torch.uint8)], -1)


def unpack_fp8(rows: torch.Tensor) -> torch.Tensor:
    """float64 values of 132-byte rows."""
    codes = rows[..., :128].contiguous().view(torch.float8_e4m3fn).double()
    return codes * rows[..., 128:].contiguous().view(torch.float32).double()


def values(pool: torch.Tensor, kind: str) -> np.ndarray:
    return (unpack_fp8(pool.cpu()) if kind == "fp8x132" else pool.cpu().double()).numpy()


class Cache:
    """A paged cache on a device (CPU tensors mirror it): keys and values of `lens` entries a
    request, one spare column and two spare pages, pages in random order."""

    def __init__(self, seed, lens, n_kv, head_dim=128, kind="bf16", device="cuda:0", extra=0):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.head_dim, self.n_kv, self.lens = kind, head_dim, n_kv, list(lens)
        B = len(self.lens)
        need = [-(-(x + extra) // PAGE) for x in self.lens]
        width = max(need + [1]) + 1
        self.n_phys = sum(need) + 2
        perm = torch.randperm(self.n_phys, generator=g).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32)
        at = 0
        for b, p in enumerate(need):
            table[b, :p] = perm[at:at + p]
            at += p
        shape = (self.n_phys, n_kv, PAGE, head_dim)
        raw = [torch.randn(*shape, generator=g) for _ in range(2)]
        pools = [pack_fp8(x) if kind == "fp8x132" else x.to(TORCH[kind]) for x in raw]
        self.device = device
        self.table, self.pools = table, pools
        self.upload()

    def upload(self):
        """The CPU mirror to the device (after a test has changed it)."""
        self.d_table = self.table.to(self.device)
        self.d_pools = [p.to(self.device) for p in self.pools]
        self.d_lens = torch.tensor(self.lens, dtype=torch.int32, device=self.device)

    def desc(self, max_len=None):
        return api.kv_desc(self.d_pools, self.kind, self.d_table, self.d_lens,
                           max(self.lens + [1]) if max_len is None else max_len, head_dim=self.head_dim)

    def rows(self, b, which):
        """float64 [len, n_kv, head_dim] and the mapped entries [len]."""
        pool = values(self.pools[which], self.kind)
        L = self.lens[b]
        out, live = np.zeros((L, self.n_kv, self.head_dim)), np.zeros(L, bool)
        for s in range(L):
            e = OC.entry(self.table[b], s, self.n_phys)
            if e:
                out[s], live[s] = pool[e[0], :, e[1]], True
        return out, live


def tree_bits(rng, n):
    """A random tree of n drafts: row i sees itself and its ancestors."""
    bits = np.zeros((n, n), bool)
    for i in range(n):
        if i:
            up = int(rng.integers(-1, i))
            if up >= 0:
                bits[i] |= bits[up]
        bits[i, i] = True
    return bits


def pack_bits(rows, words):
    """int64 [len(rows), words] of boolean rows of any length."""
    out = np.zeros((len(rows), words), np.uint64)
    for i, r in enumerate(rows):
        for j in np.flatnonzero(r):
            out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return torch.from_numpy(out.view(np.int64))


def run_attend(c, q, start, max_rows, scale, window, n_sink, mask=None, out=None, lse=None, max_len=None,
               stream=None, T=None):
    """fm_attend_window (or, with a mask, fm_attend_tree) on a Cache."""
    out = torch.full_like(q, 7.0) if out is None else out
    lse = torch.full(q.shape[:2], 7.0, device=q.device) if lse is None else lse
    d = api.attn_desc(q, "f32" if c.kind == "f32" else "bf16", out, start, max_rows, n_kv_heads=c.n_kv,
                      scale=scale, lse=lse)
    kv = c.desc(max_len)
    nb = api.fm_attend_workspace_bytes(d, kv, window, n_sink)
    ws = torch.empty(max(nb, 256), dtype=torch.uint8, device=q.device)
    if mask is None:
        api.fm_attend_window(d, kv, window, n_sink, ws, nb, stream)
    else:
        api.fm_attend_tree(d, kv, mask, mask.shape[1], window, n_sink, ws, nb, stream)
    return out, lse


def attend_oracle(c, q, ns, scale, window, n_sink, bits=None):
    """Per request: (out, lse, mag, big, seen) of the oracle."""
    res, t = [], 0
    q = q.double().cpu().numpy()
    for b, n in enumerate(ns):
        k, live = c.rows(b, 0)
        v, _ = c.rows(b, 1)
        L = c.lens[b]
        if bits is None:
            see = OC.window_rows(n, max(L, 0), window, n_sink) if L else np.zeros((n, 0), bool)
        else:
            see = OC.tree_rows(bits[b], L, window, n_sink)
        res.append(OC.attend(q[t:t + n], k, v, see & live[None], scale))
        t += n
    return [np.concatenate(x) for x in zip(*res)]


def attend_bounds(kind, D, out, lse, mag, big, seen):
    """Largest differences that rounding explains (elementwise, absolute).

    A score is a float32 dot product of D terms, scaled and shifted: off by at most
    (D + 8) 2^-24 of sum |q k| (times scale); so an exponential by twice that relatively (its own
    score and the maximum it is taken against), plus 2^-21 for exp2 and, over `seen` terms summed
    in float32, seen 2^-24 for numerator and denominator each.  bf16 and fp8 caches round every
    probability (2^-8 of sum p |v| at most) and the output (2^-8 of itself).
    """
    e = 2 * (D + 8) * 2.0 ** -24 * big + 2.0 ** -21 + 2 * seen[:, None] * 2.0 ** -24
    tol = mag * e[..., None]
    if kind != "f32":
        tol = tol + 2.0 ** -8 * (mag + np.abs(out)) * (1 + 2.0 ** -7)
    ltol = (D + 8) * 2.0 ** -24 * big + 2.0 ** -21 + seen[:, None] * 2.0 ** -24 + 2.0 ** -23 * np.abs(
        np.where(np.isfinite(lse), lse, 0))
    return tol + 1e-30, ltol


def check_attend(tag, c, got, ref, t0=0):
    out, lse, mag, big, seen = ref
    o = got[0].double().cpu().numpy()[t0:t0 + len(out)]
    l = got[1].double().cpu().numpy()[t0:t0 + len(out)]
    tol, ltol = attend_bounds(c.kind, c.head_dim, out, lse, mag, big, seen)
    assert np.array_equal(np.isneginf(l), np.isneginf(lse)), f"{tag}: empty rows"
    worst = np.max(np.abs(o - out) / tol) if out.size else 0
    fin = np.isfinite(lse)
    lw = np.max((np.abs(l - np.where(fin, lse, 0)) / ltol)[fin]) if fin.any() else 0
    assert worst <= 1 and lw <= 1, f"{tag}: out {worst:.3g} and lse {lw:.3g} of the bound"
    return worst, lw
