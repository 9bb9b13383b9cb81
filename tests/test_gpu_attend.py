"""GPU parity of fm_attend_window and fm_attend_tree against the fp64 oracle.

The bound of each element follows from the roundings (cache_util.attend_bounds).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import cache as OC
from tests import cache_util as U
from top_selection_fm_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def queries(seed, T, H, D, kind, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, D, generator=g) * std).to(U.TORCH[kind]).to(DEV)


def starts(ns):
    return torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32, device=DEV)


# kind, head_dim, heads, kv heads, lens, rows, window, sinks
CASES = [
    ("bf16", 128, 16, 2, [1000], [1], 128, 4),                    # decode, one wave a tile
    ("bf16", 128, 4, 4, [1, 2, 63, 64, 65, 0], [1, 1, 1, 1, 1, 1], 1 << 40, 0),   # lengths at page edges, an empty one
    ("bf16", 128, 8, 1, [700, 129, 1], [1, 1, 1], 64, 65),        # window of a page, sinks past a page
    ("bf16", 128, 12, 4, [513, 300], [9, 2], 100, 3),             # three heads a kv head, two rows
    ("bf16", 64, 8, 2, [333, 40, 7], [12, 16, 7], 50, 1),         # two column blocks, whole prompt
    ("bf16", 64, 2, 2, [5000], [1], 1 << 20, 0),                  # split entries, one column
    ("bf16", 128, 8, 2, [4500, 1000], [16, 3], 1 << 20, 0),       # split, two column blocks
    ("bf16", 128, 8, 2, [450, 64, 200], [200, 64, 1], 96, 5),     # 128-column blocks, ragged
    ("bf16", 64, 6, 2, [300, 257], [300, 129], 1 << 20, 0),       # plain causal prompt
    ("bf16", 128, 14, 2, [3000], [20], 2900, 10),                 # blocks and split entries
    ("fp8x132", 128, 16, 2, [900, 65], [1, 1], 300, 4),
    ("fp8x132", 128, 8, 4, [2500], [20], 1 << 20, 0),
    ("fp8x132", 128, 8, 2, [260, 100], [130, 100], 77, 2),
    ("fp8x132", 128, 16, 1, [1500], [30], 1 << 20, 0),
    ("f32", 128, 6, 2, [200, 33, 31], [1, 1, 1], 40, 2),
    ("f32", 128, 4, 1, [300], [15], 1 << 20, 0),
    ("f32", 64, 12, 4, [400, 70], [100, 70], 90, 1),
    ("f32", 128, 4, 2, [700], [70], 1 << 20, 0),
    ("f32", 64, 3, 1, [1200], [10], 1 << 20, 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_window(case):
    kind, D, H, K, lens, ns, window, sink = CASES[case]
    c = U.Cache(100 + case, lens, K, D, kind)
    q = queries(200 + case, sum(ns), H, D, kind)
    scale = D ** -0.5
    got = U.run_attend(c, q, starts(ns), max(ns), scale, window, sink)
    ref = U.attend_oracle(c, q, ns, scale, window, sink)
    print(U.check_attend(f"window {CASES[case]}", c, got, ref))
    again = U.run_attend(c, q, starts(ns), max(ns), scale, window, sink)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


TREES = [
    ("bf16", 128, 4, 1, [500], [8], 1 << 20, 0),
    ("bf16", 128, 8, 2, [127, 64, 300], [16, 1, 7], 1 << 20, 0),
    ("bf16", 128, 8, 2, [3000, 130], [64, 40], 1 << 20, 0),        # drafts across a page edge, split entries
    ("bf16", 64, 4, 2, [400, 100], [100, 77], 60, 3),               # two mask words, window and sinks
    ("fp8x132", 128, 8, 2, [600, 129], [33, 65], 1 << 20, 0),
    ("fp8x132", 128, 4, 4, [2000], [12], 500, 4),
    ("f32", 64, 4, 2, [200, 90], [33, 64], 50, 2),
    ("f32", 128, 6, 2, [300], [130], 1 << 20, 0),
]


@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree(case):
    kind, D, H, K, lens, ns, window, sink = TREES[case]
    rng = np.random.default_rng(case)
    c = U.Cache(300 + case, lens, K, D, kind)
    q = queries(400 + case, sum(ns), H, D, kind)
    bits = [U.tree_bits(rng, n) for n in ns]
    if case == 3:
        bits[0][5] = False                                          # a row that sees no draft
    words = -(-max(ns) // 64)
    rows = [np.concatenate([r, rng.random(64 * words - len(r)) < 0.5]) for x in bits for r in x]   # bits past n
    mask = U.pack_bits(rows, words).to(DEV)
    got = U.run_attend(c, q, starts(ns), max(ns), D ** -0.5, window, sink, mask=mask)
    ref = U.attend_oracle(c, q, ns, D ** -0.5, window, sink, bits=bits)
    print(U.check_attend(f"tree {TREES[case]}", c, got, ref))


def test_chain_of_drafts_is_the_window():
    """A tree that is a chain sees what the causal window sees."""
    ns = [20, 3]
    c = U.Cache(7, [400, 90], 2)
    q = queries(8, 23, 8, 128, "bf16")
    words = 1
    mask = U.pack_bits([np.arange(64) <= i for n in ns for i in range(n)], words).to(DEV)
    a = U.run_attend(c, q, starts(ns), 20, 0.1, 1 << 20, 0)
    b = U.run_attend(c, q, starts(ns), 20, 0.1, 1 << 20, 0, mask=mask)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind,H,K,ns", [("bf16", 8, 2, [1, 1, 1]), ("bf16", 8, 2, [12, 3, 5]),
                                         ("bf16", 8, 2, [100, 1, 60]), ("fp8x132", 8, 2, [1, 1, 1]),
                                         ("fp8x132", 8, 2, [100, 1, 60]), ("f32", 4, 2, [1, 1, 1]),
                                         ("f32", 4, 2, [90, 1, 70])])
def test_masked_places_may_hold_anything(kind, H, K, ns):
    """NaN, infinities and the type's extremes in every hidden entry, every page outside the
    tables, and the table's unused cells: the result is the same bits as with zeros there."""
    D, window, sink = 128, 70, 3
    lens = [300, 77, 190]
    c = U.Cache(50, lens, K, D, kind)
    q = queries(51, sum(ns), H, D, kind)
    seen = torch.zeros(c.n_phys, 64, dtype=torch.bool)
    for b, n in enumerate(ns):
        see = OC.window_rows(n, lens[b], window, sink).any(0)
        for s in np.flatnonzero(see):
            seen[c.table[b, s // 64], s % 64] = True
    base = [p.clone() for p in c.pools]
    res = []
    for fill in ("zero", "nan", "inf", "low"):
        for i, p in enumerate(base):
            x = p.clone()
            hide = ~seen[:, None, :, None].expand(*x.shape)
            if kind == "fp8x132":
                row = torch.zeros(132, dtype=torch.uint8)
                row[:128] = {"zero": 0, "nan": 0x7f, "inf": 0x7e, "low": 0xfe}[fill]
                row[128:] = torch.tensor([{"zero": 1.0, "nan": float("nan"), "inf": float("inf"),
                                           "low": 3e38}[fill]]).view(torch.uint8)
                x = torch.where(hide, row, x)
            else:
                v = {"zero": 0.0, "nan": float("nan"), "inf": float("inf"), "low": torch.finfo(x.dtype).min}[fill]
                x = torch.where(hide, torch.full_like(x, v), x)
            c.pools[i] = x
        if fill != "zero":
            c.table[c.table < 0] = {"nan": 1 << 30, "inf": -(1 << 31), "low": c.n_phys}[fill]
        c.upload()
        res.append(U.run_attend(c, q, starts(ns), max(ns), 0.09, window, sink))
    for out, lse in res[1:]:
        assert torch.equal(out, res[0][0]) and torch.equal(lse, res[0][1])
    assert bool(torch.isfinite(res[0][0].float()).all())


@pytest.mark.parametrize("ns", [[2, 2], [70, 40]])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_hidden_from_some_rows_only(kind, ns):
    """Infinities and NaN in values that some rows see and others do not reach the former alone,
    each as IEEE arithmetic has it."""
    D, window = 64, 30
    lens = [200, 100]
    c = U.Cache(60, lens, 2, D, kind)
    q = queries(61, sum(ns), 4, D, kind)
    for b in range(2):
        for s, val in ((lens[b] - 1, float("inf")), (lens[b] - 29, float("nan")), (lens[b] - 31, float("-inf"))):
            page = int(c.table[b, s // 64])
            c.pools[1][page, b, s % 64, 3 + b] = val
            c.pools[1][page, b, s % 64, 40] = -val
    c.upload()
    out, lse = U.run_attend(c, q, starts(ns), max(ns), 0.1, window, 0)
    ref = U.attend_oracle(c, q, ns, 0.1, window, 0)
    got, want = out.double().cpu().numpy(), ref[0]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.isnan(want).any() and np.array_equal(got[inf], want[inf])
    fine = np.isfinite(want)
    tol, _ = U.attend_bounds(kind, D, np.where(fine, want, 0), ref[1], np.where(fine, ref[2], 0), ref[3], ref[4])
    assert np.all(np.abs(got - want)[fine] <= tol[fine])


@pytest.mark.parametrize("ns", [[2, 2], [70, 40]])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_each_infinity_in_a_value_of_its_own(kind, ns):
    """As above, +inf, -inf and NaN in values of their own, so the infinities are seen alone."""
    D, window = 64, 30
    lens = [200, 100]
    c = U.Cache(62, lens, 2, D, kind)
    q = queries(63, sum(ns), 4, D, kind)
    for b in range(2):
        for i, (back, val) in enumerate(((1, float("inf")), (31, float("-inf")), (2, float("nan")), (30, float("inf")))):
            s = lens[b] - back
            c.pools[1][int(c.table[b, s // 64]), :, s % 64, 8 * i + b] = val
    c.upload()
    out, _ = U.run_attend(c, q, starts(ns), max(ns), 0.1, window, 0)
    want = U.attend_oracle(c, q, ns, 0.1, window, 0)[0]
    got = out.double().cpu().numpy()
    bad = ~np.isfinite(want)
    assert np.isposinf(want).any() and np.isneginf(want).any() and np.isnan(want).any()
    assert np.array_equal(got[bad], want[bad], equal_nan=True) and np.isfinite(got[~bad]).all()


def test_visible_key_nan_poisons_its_rows_only():
    c = U.Cache(70, [150], 1, 128, "bf16")
    c.pools[0][int(c.table[0, 1]), 0, 70 - 64, 5] = float("nan")     # entry 70
    c.upload()
    q = queries(71, 120, 2, 128, "bf16")                              # rows 30 .. 149
    out, lse = U.run_attend(c, q, starts([120]), 120, 0.1, 40, 0)
    bad = torch.isnan(out.float()).all(-1).all(-1).cpu().numpy()
    rows = np.arange(30, 150)
    assert np.array_equal(bad, (rows >= 70) & (rows < 110))
    assert not torch.isnan(out.float())[~torch.from_numpy(bad)].any()


def test_unmapped_pages_and_rows_outside():
    """Pages a window has left behind (-1), pages past the pool, rows before q_start[0] and
    behind q_start[B], a request without rows, and rows beyond a request's entries."""
    lens = [400, 10, 64, 200]
    c = U.Cache(80, lens, 2)
    c.table[0, 1], c.table[0, 3] = -1, c.n_phys + 5
    c.table[2, 0] = -1                                                # nothing left to see
    c.upload()
    ns = [6, 12, 2, 0]                                                # 12 rows, 10 entries: two are empty
    q = queries(81, 3 + 20 + 4, 8, 128, "bf16")
    start = starts(ns) + 3
    out, lse = U.run_attend(c, q, start, 12, 0.1, 1 << 20, 0)
    assert bool((out[:3] == 7).all()) and bool((out[23:] == 7).all()) and bool((lse[23:] == 7).all())
    assert bool((out[9:11] == 0).all()) and bool(torch.isneginf(lse[9:11]).all())
    assert bool((out[21:23] == 0).all()) and bool(torch.isneginf(lse[21:23]).all())
    c2 = U.Cache(80, [400], 2)                                        # the same pages, read on the CPU
    c2.table, c2.n_phys, c2.pools = c.table[:1], c.n_phys, c.pools
    ref = U.attend_oracle(c2, q[3:9], [6], 0.1, 1 << 20, 0)
    U.check_attend("unmapped", c2, (out[3:9], lse[3:9]), ref)
    c3 = U.Cache(80, [10], 2)
    c3.table, c3.n_phys, c3.pools = c.table[1:2], c.n_phys, c.pools
    U.check_attend("short", c3, (out[11:21], lse[11:21]), U.attend_oracle(c3, q[11:21], [10], 0.1, 1 << 20, 0))


@pytest.mark.parametrize("rows,H,K", [(1, 8, 2), (40, 8, 2)])
def test_strided_rows_and_row_bound(rows, H, K):
    """q and out as slices of wider buffers; more rows than max_rows are left as they were."""
    D = 128
    c = U.Cache(90, [300, 200], K)
    wide = queries(91, 2 * rows, H + 5, D, "bf16")
    q = wide[:, 2:2 + H]
    outw = torch.full((2 * rows, H + 3, D), 7.0, dtype=torch.bfloat16, device=DEV)
    out = outw[:, 1:1 + H]
    got = U.run_attend(c, q, starts([rows, rows]), rows, 0.1, 1 << 20, 0, out=out)
    ref = U.attend_oracle(c, q, [rows, rows], 0.1, 1 << 20, 0)
    U.check_attend("strided", c, got, ref)
    assert bool((outw[:, 0] == 7).all()) and bool((outw[:, 1 + H:] == 7).all())
    if rows > 1:
        out2, _ = U.run_attend(c, q.contiguous(), starts([rows, rows]), rows - 1, 0.1, 1 << 20, 0)
        assert bool((out2[rows - 1] == 7).all()) and bool((out2[2 * rows - 1] == 7).all())


def test_large_scores():
    """Scores of hundreds: the running maximum moves by far more than the lazy bound."""
    c = U.Cache(95, [700], 1, 128, "f32")
    ramp = torch.linspace(0.1, 6, 700)
    for s in range(700):
        c.pools[0][int(c.table[0, s // 64]), 0, s % 64] *= ramp[s]
    c.upload()
    q = queries(96, 40, 2, 128, "f32", std=6.0)
    got = U.run_attend(c, q, starts([40]), 40, 128 ** -0.5, 1 << 20, 0)
    ref = U.attend_oracle(c, q, [40], 128 ** -0.5, 1 << 20, 0)
    assert np.max(np.abs(ref[1])) > 50
    U.check_attend("large", c, got, ref)


def test_on_another_stream():
    c = U.Cache(97, [3000], 2)
    q = queries(98, 2, 8, 128, "bf16")
    a = U.run_attend(c, q, starts([2]), 2, 0.1, 1 << 20, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    st = starts([2])
    torch.cuda.synchronize()
    U.run_attend(c, q, st, 2, 0.1, 1 << 20, 0, out=out, lse=lse, stream=s)
    s.synchronize()
    assert torch.equal(out, a[0]) and torch.equal(lse, a[1])


def test_graph_replays():
    """Captured once and replayed with other eager work between: the eager bits each time."""
    c = U.Cache(99, [3000, 100], 2, 128, "fp8x132")
    q = queries(99, 10, 8, 128, "bf16")
    st = starts([5, 5])
    ref = U.run_attend(c, q, st, 5, 0.1, 2000, 4)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    d = api.attn_desc(q, "bf16", out, st, 5, n_kv_heads=2, scale=0.1, lse=lse)
    kv = c.desc()
    nb = api.fm_attend_workspace_bytes(d, kv, 2000, 4)
    ws = torch.empty(max(nb, 256), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.fm_attend_window(d, kv, 2000, 4, ws, nb)
    for i in range(4):
        out.fill_(float("nan"))
        ws.fill_(255)
        torch.randn(1 << 18, device=DEV).sum()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1]), i


@pytest.mark.parametrize("kind,ns", [("bf16", [20, 75]), ("bf16", [7, 72]), ("fp8x132", [150, 200]), ("f32", [20, 75])])
@pytest.mark.parametrize("window", [1 << 40, (1 << 31) - 1, 9])
def test_more_rows_than_entries(kind, ns, window):
    """Rows and drafts before entry 0: rows see what the formula leaves, whatever the window."""
    lens = [3, 70]
    c = U.Cache(120, lens, 2, 128, kind)
    q = queries(121, sum(ns), 4, 128, kind)
    got = U.run_attend(c, q, starts(ns), max(ns), 0.1, window, 1)
    U.check_attend("rows", c, got, U.attend_oracle(c, q, ns, 0.1, window, 1))
    bits = [U.tree_bits(np.random.default_rng(b), n) for b, n in enumerate(ns)]
    words = -(-max(ns) // 64)
    mask = U.pack_bits([r for x in bits for r in x], words).to(DEV)
    got = U.run_attend(c, q, starts(ns), max(ns), 0.1, window, 1, mask=mask)
    U.check_attend("drafts", c, got, U.attend_oracle(c, q, ns, 0.1, window, 1, bits=bits))


@pytest.mark.parametrize("kind,H,K,ns", [("bf16", 1024, 1, [1, 2]), ("fp8x132", 1024, 2, [2, 1]),
                                         ("f32", 1024, 1, [2, 1]), ("bf16", 1024, 1024, [2, 1])])
def test_most_heads(kind, H, K, ns):
    """More heads a kv head than a workgroup has columns, and as many kv heads."""
    c = U.Cache(130, [150, 40], K, 128 if kind == "fp8x132" else 64, kind)
    q = queries(131, sum(ns), H, c.head_dim, kind)
    got = U.run_attend(c, q, starts(ns), max(ns), 0.1, 100, 2)
    U.check_attend("heads", c, got, U.attend_oracle(c, q, ns, 0.1, 100, 2))


@pytest.mark.parametrize("kind,ns", [("bf16", [1]), ("bf16", [40]), ("fp8x132", [1]), ("fp8x132", [40]), ("f32", [1]),
                                     ("f32", [40])])
def test_long_table_of_unmapped_pages(kind, ns):
    """The longest lengths there are, all but the first and last pages unmapped."""
    c = U.Cache(140, [128], 2, 128, kind)
    L = (1 << 31) - 1
    cells = (L + 63) // 64
    small = [int(x) for x in c.table[0, :2]]
    q = queries(141, ns[0], 4, 128, kind)
    c.d_table = torch.full((1, cells), -1, dtype=torch.int32, device=DEV)
    c.d_table[0, 0], c.d_table[0, cells - 1] = small[0], small[1]
    c.d_lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    got = U.run_attend(c, q, starts(ns), ns[0], 0.1, 64, 10, max_len=L)
    # the same entries with one unmapped page between them: the last page ends an entry short
    c.table, c.lens = torch.tensor([[small[0], -1, small[1]]], dtype=torch.int32), [191]
    U.check_attend("long", c, got, U.attend_oracle(c, q, ns, 0.1, 64, 10))


@pytest.mark.parametrize("kind,D,ns,lens,window", [
    ("bf16", 64, [200, 1, 0, 77, 150], [1100, 1300, 900, 1090, 200], 1 << 20),
    ("fp8x132", 128, [200, 1, 0, 77, 150], [1100, 1300, 900, 1090, 200], 1 << 20),
    ("f32", 64, [100, 1, 0, 77, 50], [700, 800, 600, 90, 60], 1 << 20),
    ("bf16", 64, [100] * 9, [1030] * 9, 1 << 20),                 # alike: every block of one length but the last ones
    ("bf16", 64, [24] * 35 + [0, 1], [64 * i + 5 for i in range(37)], 1 << 20),   # trees and windows of one block each
    ("f32", 64, [20] * 30, [25 * i for i in range(30)], 1 << 20)])
def test_ragged_batches(kind, D, ns, lens, window):
    """Enough blocks of unlike lengths that their order matters: each is worked on, once."""
    H, K = 64, 8
    c = U.Cache(150, lens, K, D, kind)
    q = queries(151, sum(ns), H, D, kind)

    def check(tag, got, bits=None):
        pools = c.pools
        for k in (0, 5):                                             # the oracle is slow: two kv heads of eight
            c.pools, c.n_kv = [p[:, k:k + 1] for p in pools], 1
            part = slice(8 * k, 8 * k + 8)
            U.check_attend(f"{tag}, kv head {k}", c, (got[0][:, part], got[1][:, part]),
                           U.attend_oracle(c, q[:, part], ns, D ** -0.5, window, 0, bits=bits))
        c.pools, c.n_kv = pools, K

    check("ragged", U.run_attend(c, q, starts(ns), max(ns), D ** -0.5, window, 0))
    if max(ns) <= 64:
        bits = [U.tree_bits(np.random.default_rng(b), n) for b, n in enumerate(ns)]
        mask = U.pack_bits([r for x in bits for r in x], 1).to(DEV)
        check("ragged trees", U.run_attend(c, q, starts(ns), max(ns), D ** -0.5, window, 0, mask=mask), bits)


@pytest.mark.parametrize("ns", [[1, 2], [70, 40]])
def test_wild_scales_seen_by_some_rows(ns):
    """fp8 values whose scale is an infinity or NaN, and codes that are NaN, reach the rows that see
    them alone, each as code times scale is in IEEE arithmetic."""
    lens, window = [200, 100], 30
    c = U.Cache(160, lens, 2, 128, "fp8x132")
    q = queries(161, sum(ns), 4, 128, "bf16")
    for b in range(2):
        for h, (back, scale) in enumerate(((1, float("inf")), (29, float("-inf")))):
            s = lens[b] - back
            row = c.pools[1][int(c.table[b, s // 64]), h, s % 64]
            row[128:] = torch.tensor([scale]).view(torch.uint8)
            row[5] = 0                                               # 0 inf
        s = lens[b] - 31
        c.pools[1][int(c.table[b, s // 64]), 0, s % 64, 7] = 0x7f
        s = lens[b] - 2
        c.pools[1][int(c.table[b, s // 64]), 1, s % 64, 128:] = torch.tensor([float("nan")]).view(torch.uint8)
    c.upload()
    out, lse = U.run_attend(c, q, starts(ns), max(ns), 0.1, window, 0)
    want = U.attend_oracle(c, q, ns, 0.1, window, 0)
    got, bad = out.double().cpu().numpy(), ~np.isfinite(want[0])
    assert np.isposinf(want[0]).any() and np.isneginf(want[0]).any() and np.isnan(want[0]).any()
    assert np.array_equal(got[bad], want[0][bad], equal_nan=True) and np.isfinite(got[~bad]).all()
    assert bool(torch.isfinite(lse).all())
