"""GPU parity of the page calls (fm_cache_fork / _grow / _free / _compact) with the oracle, which
does them one page at a time: tables, lengths, references, the stack and every byte are equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import cache as OC
from top_selection_fm_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Both:
    """The same cache on the device and in the oracle."""

    def __init__(self, seed, B, N, width, pools=((2, 132), (1, 4), (3, 48))):
        rng = np.random.default_rng(seed)
        arr = [rng.integers(0, 256, (N, h, 64, row), dtype=np.uint8) for h, row in pools]
        self.o = OC.Pages(arr, np.full((B, width), -1, np.int32), np.zeros(B, np.int32), np.zeros(N, np.int32),
                          rng.permutation(N).astype(np.int32), N)
        dev = lambda a: torch.from_numpy(np.array(a)).to(DEV)  # noqa: E731
        self.pools = [dev(p) for p in arr]
        self.table, self.lens, self.ref, self.free = (dev(x) for x in (self.o.table, self.o.lens, self.o.ref, self.o.free))
        self.n_free = dev(np.array([N], np.int32))
        self.d = api.cache_desc(self.pools, self.table, self.lens, self.ref, self.free, self.n_free)

    def call(self, name, *lists, deep=False, keep=None, stream=None):
        """One call on both sides; everything is compared."""
        n = len(lists[0])
        ints = [None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV) for x in lists]
        ok = torch.full((n + 1,), 9, dtype=torch.int32, device=DEV)
        nb = api.fm_cache_workspace_bytes(self.d, n)
        ws = torch.full((nb,), 255, dtype=torch.uint8, device=DEV)
        if name == "fork":
            api.fm_cache_fork(self.d, ints[0], ints[1], n, deep, ok, ws, nb, stream)
            want = self.o.fork(*lists, deep)
        elif name == "grow":
            api.fm_cache_grow(self.d, ints[0], ints[1], n, ok, ws, nb, stream)
            want = self.o.grow(*lists)
        elif name == "free":
            api.fm_cache_free(self.d, ints[0], ints[1], n, ok, stream)
            want = self.o.free_requests(*lists)
        else:
            width = max([len(k) for k in keep] + [1]) + 1
            kk = torch.tensor([list(k) + [-1] * (width - len(k)) for k in keep], dtype=torch.int32, device=DEV)
            cnt = torch.tensor([len(k) for k in keep], dtype=torch.int32, device=DEV)
            api.fm_cache_compact(self.d, ints[0], ints[1], kk, width, cnt, n, ok, stream)
            want = self.o.compact(lists[0], lists[1], keep, [len(k) for k in keep])
        torch.cuda.synchronize()
        assert ok.tolist() == want + [9], (name, lists)
        self.same(name)
        return want

    def same(self, what):
        o = self.o
        assert int(self.n_free) == o.n_free, what
        for got, ref in ((self.table, o.table), (self.lens, o.lens), (self.ref, o.ref)):
            assert np.array_equal(got.cpu().numpy(), ref), what
        assert np.array_equal(self.free.cpu().numpy()[:o.n_free], o.free[:o.n_free]), what
        for l, (p, q) in enumerate(zip(self.pools, o.pools)):
            held = o.ref > 0                                # what a free page holds is nobody's
            assert np.array_equal(p.cpu().numpy()[held], q[held]), f"{what}: pool {l}"
        use = np.zeros_like(o.ref)
        for b in range(len(o.lens)):
            for c in range(-(-int(o.lens[b]) // 64)):
                if 0 <= o.table[b, c] < len(use):
                    use[o.table[b, c]] += 1
        assert np.array_equal(use, o.ref), what             # references are cells in use
        assert o.n_free == (use == 0).sum()


def test_life_of_a_few_requests():
    c = Both(1, 6, 24, 6)
    assert c.call("grow", [0, 1, 2], [130, 64, 1]) == [1, 1, 1]
    assert c.call("fork", [0, 1, 2, 5], [3, 4, 5, 2]) == [1, 1, 1, 0]   # 2 is not empty
    assert c.call("grow", [3, 0], [140, 131]) == [1, 1]
    assert c.call("compact", [3, 1], [128, 0], keep=[[130, 133, 139], [0, 1, 5]]) == [1, 0]   # 1's page is shared
    assert c.call("free", [4], None) == [1]
    assert c.call("compact", [1], [0], keep=[[3, 9, 63]]) == [1]
    assert c.call("free", [0, 3, 1, 2, 5], None) == [1] * 5
    assert c.o.n_free == 24


def test_shared_pages_are_copied_before_growth():
    """Cut inside a shared page, both holders grow in one call: each gets a copy and the page,
    which nobody holds any more, goes back."""
    c = Both(2, 4, 12, 4)
    c.call("grow", [0], [128])
    c.call("fork", [0], [1])
    c.call("free", [0, 1], [100, 90])
    c.call("grow", [0, 1], [101, 91])
    assert c.o.table[0, 1] != c.o.table[1, 1]
    c.call("fork", [0], [2], deep=True)
    c.call("compact", [0], [10], keep=[[20, 70, 100]])                   # its first page is shared
    c.call("free", [1], [0])
    assert c.call("compact", [0], [10], keep=[[20, 70, 100]]) == [1]


def test_refusals_on_the_device():
    c = Both(3, 4, 10, 3)
    assert c.call("grow", [0, 0, -1, 4, 1, 2], [64, 128, 1, 1, 193, -5]) == [1, 0, 0, 0, 0, 0]
    assert c.call("grow", [0], [63]) == [0]
    assert c.call("free", [0, 0, 1, 7], [65, 0, -1, 0]) == [0, 0, 0, 0]  # the first names 0, and is refused
    assert c.call("fork", [0, 0, 1, 9], [0, 1, 1, 2]) == [0, 1, 0, 0]
    for keep in ([5, 5], [6, 5], [64], [-1], [1, 2, 200]):
        assert c.call("compact", [0], [0], keep=[keep]) == [0]
    assert c.call("compact", [0], [65], keep=[[]]) == [0]
    assert c.call("compact", [0, 0], [64, 0], keep=[[], [1]]) == [1, 0]


@pytest.mark.parametrize("deep", [False, True])
def test_not_enough_pages(deep):
    """The first entry that does not fit is refused, and every valid one after it."""
    c = Both(4, 8, 9, 4)
    assert c.call("grow", [0, 1], [65, 130]) == [1, 1]                   # 5 of 9
    assert c.call("grow", [2, 3, 4, 5], [64, 200, 1, 0]) == [1, 0, 0, 0]
    assert c.call("fork", [0, 2, 1, 0, 1], [3, 4, 5, 6, 7], deep=deep) == ([1, 1, 0, 0, 0] if deep else [1, 1, 1, 1, 0])


def test_verdicts_come_before_releases():
    """Two holders of a page compact in one call: the page is shared when the call begins, so the
    one that writes it is refused although the other gives it up."""
    c = Both(5, 3, 12, 4)
    c.call("grow", [0], [128])
    c.call("fork", [0], [1])
    assert c.call("compact", [0, 1], [64, 0], keep=[[], [3, 7]]) == [1, 0]
    assert c.call("compact", [1], [64], keep=[[70, 71]]) == [1]


def test_long_compaction_in_place():
    """Chunks that overlap: one of every three entries of 20 pages, and all but the first."""
    for seed, keep in ((6, list(range(2, 1280, 3))), (7, list(range(1, 1280))), (8, [0, 1, 2] + list(range(700, 1270)))):
        c = Both(seed, 2, 50, 20, pools=((1, 16), (2, 256), (1, 20)))
        c.call("grow", [1, 0], [1280, 1280])
        assert c.call("compact", [1], [0], keep=[keep]) == [1]


def test_wide_rows():
    """Rows past a workgroup's reach move in columns."""
    c = Both(9, 1, 4, 3, pools=((1, 4 * 1100), (1, 16 * 1030)))
    c.call("grow", [0], [130])
    assert c.call("compact", [0], [3], keep=[[5, 6, 64, 128]]) == [1]


def test_many_requests():
    """More entries than a workgroup has threads, more pages than one pass over the bitmap."""
    B = 2500
    c = Both(10, B, 40000, 3, pools=((1, 4),))
    rng = np.random.default_rng(11)
    lens = rng.integers(0, 150, B).tolist()
    order = rng.permutation(B).tolist()
    c.call("grow", order, [lens[b] for b in order])
    c.call("free", order[:1700], [lens[b] // 2 for b in order[:1700]])
    gone = order[1000:2200]
    c.call("free", gone, None)
    c.call("fork", order[:1000], gone[:1000])
    c.call("fork", order[:150], gone[1000:1150], deep=True)


@pytest.mark.parametrize("seed", range(6))
def test_random_histories(seed):
    rng = np.random.default_rng(100 + seed)
    B, width = 9, 5
    c = Both(200 + seed, B, 30, width, pools=((1, 132), (2, 16)))
    for step in range(25):
        n = int(rng.integers(1, 7))
        req = rng.integers(-1, B + 1, n).tolist()
        lens = c.o.lens
        at = lambda r: int(lens[r]) if 0 <= r < B else 0  # noqa: E731
        op = rng.choice(["grow", "grow", "fork", "fork", "free", "compact", "compact"])
        if op == "grow":
            c.call("grow", req, [at(r) + int(rng.integers(-3, 120)) for r in req])
        elif op == "fork":
            c.call("fork", rng.integers(-1, B + 1, n).tolist(), req, deep=bool(rng.random() < 0.3))
        elif op == "free":
            c.call("free", req, None if rng.random() < 0.3 else [int(rng.integers(-1, at(r) + 2)) for r in req])
        else:
            start = [int(rng.integers(0, at(r) + 1)) for r in req]
            keep = [sorted(rng.choice(np.arange(s, max(s + 1, at(r))), min(at(r) - s, int(rng.integers(0, 9))),
                                      replace=False).tolist()) if at(r) > s else [] for r, s in zip(req, start)]
            c.call("compact", req, start, keep=keep)


def test_graph_replays_and_another_stream():
    """A step (grow, compact, free, fork) captured once: each replay does what the oracle does."""
    c = Both(12, 4, 20, 4)
    c.call("grow", [0, 1], [100, 70])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    req, more, cut, start, keep, cnt = i32([0, 1]), i32([140, 100]), i32([90, 65]), i32([100, 70]), i32([[110, 139], [71, 90]]), i32([2, 2])
    src, dst = i32([0, 1]), i32([2, 3])
    nb = api.fm_cache_workspace_bytes(c.d, 2)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    ok = torch.zeros(5, 2, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.fm_cache_grow(c.d, req, more, 2, ok[0], ws, nb)
        api.fm_cache_compact(c.d, req, start, keep, 2, cnt, 2, ok[1])
        api.fm_cache_free(c.d, dst, None, 2, ok[2])
        api.fm_cache_fork(c.d, src, dst, 2, False, ok[3], ws, nb)
        api.fm_cache_free(c.d, req, start, 2, ok[4])
    for i in range(4):
        ws.fill_(255)
        torch.randn(1 << 16, device=DEV).sum()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = [c.o.grow([0, 1], [140, 100]), c.o.compact([0, 1], [100, 70], [[110, 139], [71, 90]], [2, 2]),
                c.o.free_requests([2, 3]), c.o.fork([0, 1], [2, 3], False), c.o.free_requests([0, 1], [100, 70])]
        assert ok.tolist() == want
        c.same(f"replay {i}")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.call("grow", [0], [120], stream=s)
