"""GPU parity of fm_qk_norm_rope against the fp64 oracle.

Bounds: everything up to the store is float32.  The norm is a sum of D squares, a square root, a
division and two products, each off by at most half a unit: (D + 8) 2^-24 of the value is more
than they can add up to; the angle is reduced in float64 and its sine and cosine are off by at
most 2^-21 (2^-24 of a turn times 2 pi, and the functions' own error), so a rotated value by
2^-21 + 4 2^-24 of |a| + |b|.  bf16 adds half a unit of the result, 2^-8; an e4m3 code of x / scale
is the nearest code to a quotient that is off by the above: x' and code x scale differ by half a
code step (2^-4 of the value, or 2^-10 of the scale below the normal codes) plus that.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import cache as OC
from oracle.encoder import yarn_inv_freq
from tests import cache_util as U
from top_selection_fm_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROPE = dict(rope_base=160000.0, rope_factor=16.0, rope_orig_len=65536, beta_fast=32.0, beta_slow=1.0)


def freqs(rope_dim, **kw):
    r = dict(ROPE, **kw)
    return yarn_inv_freq(rope_dim, r["rope_base"], r["rope_factor"], r["rope_orig_len"], r["beta_fast"],
                         r["beta_slow"]) if rope_dim else np.zeros(0)


def bound(ref, weighted, kind, D, first, half, halves):
    """Elementwise bound of a turned head [.., D] (see the module's text)."""
    a = np.abs(ref)
    pair = a.copy()
    if half:
        x, y = (first + np.arange(half), first + half + np.arange(half)) if halves else \
            (first + 2 * np.arange(half), first + 2 * np.arange(half) + 1)
        r = np.hypot(ref[..., x], ref[..., y]) * np.sqrt(2)     # |a| + |b| <= sqrt 2 of the pair's length
        pair[..., x] = pair[..., y] = r
    t = pair * ((D + 8) * 2.0 ** -24 + (2.0 ** -21 + 4 * 2.0 ** -24 if half else 0))
    return t + (a * 2.0 ** -8 if kind == "bf16" else 0) + 1e-30


# kind, cache kind, D, T, heads, kv heads, rope_dim, first, halves, norm
CASES = [
    ("bf16", "bf16", 128, 1, 8, 2, 64, 64, False, True),
    ("bf16", "bf16", 128, 33, 12, 4, 128, 0, True, True),
    ("bf16", "fp8x132", 128, 40, 16, 2, 64, 64, False, True),
    ("bf16", "fp8x132", 128, 1100, 4, 1, 128, 0, True, True),
    ("bf16", "bf16", 64, 70, 7, 7, 32, 16, True, True),
    ("bf16", "bf16", 64, 5, 1, 1, 2, 62, False, False),
    ("bf16", None, 128, 19, 6, 3, 64, 0, False, True),
    ("bf16", "bf16", 128, 3, 0, 2, 0, 0, False, True),
    ("f32", "f32", 128, 37, 6, 2, 128, 0, False, True),
    ("f32", "f32", 64, 9, 3, 1, 48, 8, True, True),
    ("f32", "f32", 128, 1030, 2, 2, 64, 64, True, False),
    ("f32", None, 64, 4, 5, 0, 64, 0, True, True),
]


def setup(seed, T, H, K, D, dt):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(T, H + 2 * K, D, generator=g) * 2).to(dt)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dt) for _ in range(2)]
    pos = torch.randint(0, 3_000_000, (T,), generator=g).to(torch.int32)
    return g, qkv, w, pos


@pytest.mark.parametrize("case", range(len(CASES)))
def test_norm_rope_and_store(case):
    kind, ck, D, T, H, K, R, first, halves, norm = CASES[case]
    dt = U.TORCH[kind]
    g, qkv, w, pos = setup(500 + case, T, H, K, D, dt)
    B = 3
    lens = [T + 70, T // 2 + 65, 64]
    d = qkv.to(DEV)
    wd = [x.to(DEV) if norm else None for x in w]
    qo = torch.full((T, H, D), 7.0, dtype=dt, device=DEV) if H else None
    ko = torch.full((T, K, D), 7.0, dtype=dt, device=DEV) if K else None
    kw = dict(rope_dim=R, rope_first=first, rope_halves=halves, rms_eps=1e-5, k_out=ko, **ROPE)
    q, k, v = d[:, :H] if H else None, d[:, H:H + K] if K else None, d[:, H + K:] if K and ck else None
    c = None
    if ck:
        c = U.Cache(600 + case, lens, K, D, ck)
        c.table[1, 0] = -1                                              # a page the window has left
        c.upload()
        before = [p.clone() for p in c.pools]
        # every row an entry of its own; some out of range, in no request, or in no page
        cells = [(b, s) for b in range(B) for s in range(lens[b])]
        pick = torch.randperm(len(cells), generator=g)[:T].tolist()
        req = torch.tensor([cells[i][0] for i in pick], dtype=torch.int32)
        slot = torch.tensor([cells[i][1] for i in pick], dtype=torch.int32)
        if T > 8:
            req[1], req[2], slot[3], slot[4] = -1, B, -1, lens[req[4]]
        kw.update(row_req=req.to(DEV), slot=slot.to(DEV))
    desc = api.qk_desc(q, k, v, kind, qo, wd[0], wd[1], pos.to(DEV), **kw)
    api.fm_qk_norm_rope(desc, None if c is None else c.desc())
    torch.cuda.synchronize()
    assert torch.equal(d.cpu(), qkv)                                    # inputs untouched
    x = qkv.double().numpy()
    inv = freqs(R)
    wn = [y.double().numpy() if norm else None for y in w]
    refs = [OC.qk_norm_rope(x[:, :H], wn[0], 1e-5, pos.numpy(), inv, first, halves),
            OC.qk_norm_rope(x[:, H:H + K], wn[1], 1e-5, pos.numpy(), inv, first, halves)]
    for got, ref in ((qo, refs[0]), (ko, refs[1])):
        if got is not None:
            tol = bound(ref, norm, kind, D, first, R // 2, halves)
            worst = np.max(np.abs(got.double().cpu().numpy() - ref) / tol)
            assert worst <= 1, f"{CASES[case]}: {worst:.3g} of the bound"
    if c is None:
        return
    want = [p.clone() for p in before]
    stored = np.zeros((c.n_phys, 64), bool)
    for t in range(T):
        r, s = int(req[t]), int(slot[t])
        e = OC.entry(c.table[r], s, c.n_phys) if 0 <= r < B and 0 <= s < lens[r] else None
        if e is None:
            continue
        stored[e] = True
        for which, ref in ((0, refs[1][t]), (1, x[t, H + K:])):
            got = U.values(c.d_pools[which][e[0], :, e[1]], ck)
            base = bound(ref, norm, "f32" if ck != "bf16" else "bf16", D, first, R // 2 if which == 0 else 0, halves)
            if which == 1 and ck != "fp8x132":
                assert np.array_equal(got, ref)                         # values are copied
                continue
            if ck == "fp8x132":
                scale = np.abs(ref).max(-1, keepdims=True) / 448
                base = base + np.abs(ref) * 2.0 ** -4 * (1 + 2.0 ** -10) + scale * 2.0 ** -10 * (1 + 2.0 ** -10)
                gs = c.d_pools[which][e[0], :, e[1], 128:].contiguous().view(torch.float32).double().cpu().numpy()
                assert np.all(np.abs(gs - scale) <= scale * 2.0 ** -16)
            assert np.all(np.abs(got - ref) <= base), (t, which)
    for which in range(2):                                              # nothing else was written
        got = c.d_pools[which].cpu()
        hole = torch.from_numpy(~stored)[:, None, :, None].expand(*got.shape)
        assert torch.equal(got[hole], want[which][hole])


def test_in_place_and_rows_by_default():
    """Outputs in place; without row_req and slot, row t is request t and its entry is pos[t]."""
    T, H, K, D = 3, 4, 2, 128
    _, qkv, w, _ = setup(700, T, H, K, D, torch.bfloat16)
    c = U.Cache(701, [5, 130, 64], K)
    pos = torch.tensor([4, 129, 64], dtype=torch.int32)                 # the last is past its request
    d, wd = qkv.to(DEV), [x.to(DEV) for x in w]
    sep = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    api.fm_qk_norm_rope(api.qk_desc(d[:, :H], d[:, H:H + K], d[:, H + K:], "bf16", sep, *wd, pos.to(DEV)), c.desc())
    stored = [p.clone() for p in c.d_pools]
    k_ref = stored[0][int(c.table[1, 2]), :, 1].clone()
    e = d.clone()
    api.fm_qk_norm_rope(api.qk_desc(e[:, :H], e[:, H:H + K], None, "bf16", e[:, :H], *wd, pos.to(DEV),
                                    k_out=e[:, H:H + K]), None)
    torch.cuda.synchronize()
    assert torch.equal(e[:, :H], sep) and torch.equal(e[1, H:H + K], k_ref) and torch.equal(e[:, H + K:], d[:, H + K:])
    assert torch.equal(stored[0][int(c.table[2, 0])].cpu(), c.pools[0][int(c.table[2, 0])])


def test_rows_of_zeros_and_extremes():
    """A head of zeros stays zeros (scale 1 in a 132-byte row); the type's largest values neither
    overflow the norm nor leave the code range."""
    T, K, D = 4, 1, 128
    x = torch.zeros(T, 2 * K, D)
    x[1] = 3e38
    x[2, :, ::2] = 1e-30
    x[3, :, 5] = -448.0
    d = x.to(torch.bfloat16).to(DEV)
    c = U.Cache(702, [T], K, D, "fp8x132")
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    api.fm_qk_norm_rope(api.qk_desc(None, d[:, :K], d[:, K:], "bf16", None, None, None, pos, rope_dim=0, rope_first=0),
                        c.desc())
    torch.cuda.synchronize()
    page = int(c.table[0, 0])
    for p in c.d_pools:
        rows = p[page, 0, :T].cpu()
        scale = rows[:, 128:].contiguous().view(torch.float32)[:, 0]
        assert scale[0] == 1 and not rows[0, :128].any()
        assert bool((rows[1, :128] == 0x7e).all()) and torch.isfinite(scale).all()
        assert rows[3, 5] == 0xfe and scale[3] == 1
        back = U.unpack_fp8(rows)[2]
        assert torch.allclose(back[::2], torch.full((64,), 1e-30, dtype=torch.float64), rtol=2 ** -7)


@pytest.mark.parametrize("factor", [1.0, 16.0])
def test_far_positions(factor):
    """Positions of millions: the angle is formed in 64 bits."""
    T, D = 6, 128
    _, x, _, _ = setup(703, T, 2, 0, D, torch.float32)
    pos = torch.tensor([0, 1, 999_999, 8_388_609, 1 << 30, (1 << 31) - 1], dtype=torch.int32)
    out = torch.empty(T, 2, D, device=DEV)
    api.fm_qk_norm_rope(api.qk_desc(x.to(DEV), None, None, "f32", out, None, None, pos.to(DEV), rope_dim=D,
                                    rope_factor=factor), None)
    ref = OC.qk_norm_rope(x.double().numpy(), None, 0, pos.numpy(), freqs(D, rope_factor=factor), 0, False)
    tol = bound(ref, False, "f32", D, 0, D // 2, False)
    assert np.max(np.abs(out.double().cpu().numpy() - ref) / tol) <= 1


def test_graph_replays():
    T, H, K, D = 20, 8, 2, 128
    _, qkv, w, pos = setup(704, T, H, K, D, torch.bfloat16)
    c = U.Cache(705, [200], K, D, "fp8x132")
    d, wd = qkv.to(DEV), [x.to(DEV) for x in w]
    qo = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    slot = torch.arange(100, 100 + T, dtype=torch.int32, device=DEV)
    desc = api.qk_desc(d[:, :H], d[:, H:H + K], d[:, H + K:], "bf16", qo, *wd, pos.to(DEV), slot=slot)
    kv = c.desc()
    api.fm_qk_norm_rope(desc, kv)
    ref = [qo.clone()] + [p.clone() for p in c.d_pools]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.fm_qk_norm_rope(desc, kv)
    for _ in range(4):
        for t in [qo] + c.d_pools:
            t.zero_()
        torch.randn(1 << 16, device=DEV).sum()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, ref[0])
        for p, r in zip(c.d_pools, ref[1:]):
            for s in range(100, 100 + T):
                page = int(c.table[0, s // 64])
                assert torch.equal(p[page, :, s % 64], r[page, :, s % 64])
