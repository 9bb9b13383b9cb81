"""The paged-cache calls as a serving loop runs them: prompt, selection-free decode with a window,
a drafted tree, its accepted path kept, a fork that goes its own way, and the end of a request.

After each step the device's cache is read back through its own tables; every attention result is
compared with the fp64 oracle over those rows (the rounding bound of cache_util), and the rows
themselves with the fp64 norm and rotation of the tokens that should be there.
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
H, K, D, R = 8, 2, 128, 64
SCALE = D ** -0.5


class Server:
    """Two attention layers and an index pool over one set of pages."""

    def __init__(self, kind, B=4, pages=40, width=8):
        i32 = lambda *a: torch.zeros(*a, dtype=torch.int32, device=DEV)  # noqa: E731
        row = {"bf16": (D, torch.bfloat16), "fp8x132": (132, torch.uint8), "f32": (D, torch.float32)}[kind]
        self.kind = kind
        self.pools = [torch.zeros(pages, K, 64, row[0], dtype=row[1], device=DEV) for _ in range(4)]
        self.index = torch.zeros(pages, 64, 132, dtype=torch.uint8, device=DEV)
        self.table, self.lens = torch.full((B, width), -1, dtype=torch.int32, device=DEV), i32(B)
        self.ref, self.free = i32(pages), torch.randperm(pages, device=DEV).to(torch.int32)
        self.n_free = torch.full((1,), pages, dtype=torch.int32, device=DEV)
        self.cache = api.cache_desc(self.pools + [self.index], self.table, self.lens, self.ref, self.free, self.n_free)
        self.kv = api.kv_desc(self.pools, kind, self.table, self.lens, 64 * width)
        self.tokens = [[] for _ in range(B)]          # per request: (token id, position) of every entry
        nb = api.fm_cache_workspace_bytes(self.cache, 16)
        self.ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
        dt = U.TORCH[kind]
        g = torch.Generator().manual_seed(9)
        self.qkv = torch.randn(2, 1000, (H + 2 * K), D, generator=g).to(dt).to(DEV)   # of token ids, per layer
        self.norm = [(1 + 0.2 * torch.randn(D, generator=g)).to(dt).to(DEV) for _ in range(2)]
        self.inv = yarn_inv_freq(R, 160000.0, 16.0, 65536, 32.0, 1.0)

    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def page(self, call, *a):
        ok = self.ints([0] * 16)
        getattr(api, call)(self.cache, *a, ok=ok, **({"ws": self.ws, "ws_bytes": self.ws.numel()}
                                                    if call in ("fm_cache_fork", "fm_cache_grow") else {}))
        n = [x for x in a if isinstance(x, int)][0 if call != "fm_cache_compact" else 1]
        assert ok.tolist()[:n] == [1] * n, call

    def step(self, new, bits=None, window=1 << 20, sink=0):
        """new: {request: [(token id, position)]}: grown, written and attended on both layers."""
        reqs = sorted(new)
        self.page("fm_cache_grow", self.ints(reqs), self.ints([len(self.tokens[b]) + len(new[b]) for b in reqs]), len(reqs))
        rows = [(b, len(self.tokens[b]) + i, t, p) for b in reqs for i, (t, p) in enumerate(new[b])]
        for b in reqs:
            self.tokens[b] += new[b]
        B = len(self.tokens)
        start = np.concatenate([[0], np.cumsum([len(new.get(b, [])) for b in range(B)])])
        ids = torch.tensor([r[2] for r in rows], device=DEV)
        req, slot, pos = (self.ints([r[i] for r in rows]) for i in (0, 1, 3))
        d_start, most = self.ints(start.tolist()), max(len(v) for v in new.values())
        for layer in range(2):
            x = self.qkv[layer][ids].contiguous()
            kw = dict(layer=layer, row_req=req, slot=slot, rope_dim=R)
            kind = "f32" if self.kind == "f32" else "bf16"
            api.fm_qk_norm_rope(api.qk_desc(x[:, :H], x[:, H:H + K], x[:, H + K:], kind, x[:, :H], *self.norm, pos, **kw),
                                self.kv)
            q, out = x[:, :H].contiguous(), torch.empty(len(rows), H, D, dtype=x.dtype, device=DEV)
            lse = torch.empty(len(rows), H, device=DEV)
            d = api.attn_desc(q, kind, out, d_start, most, n_kv_heads=K, scale=SCALE, lse=lse, layer=layer)
            nb = api.fm_attend_workspace_bytes(d, self.kv, window, sink)
            ws = torch.empty(max(nb, 256), dtype=torch.uint8, device=DEV)
            if bits is None:
                api.fm_attend_window(d, self.kv, window, sink, ws, nb)
            else:
                mask = U.pack_bits([r for b in reqs for r in bits[b]], 1).to(DEV)
                api.fm_attend_tree(d, self.kv, mask, 1, window, sink, ws, nb)
            torch.cuda.synchronize()
            self.check(layer, reqs, new, q, out, lse, bits, window, sink)

    def check(self, layer, reqs, new, q, out, lse, bits, window, sink):
        at = 0
        kv = [U.values(p, self.kind) for p in self.pools[2 * layer:2 * layer + 2]]
        table = self.table.cpu().numpy()
        assert self.lens.tolist() == [len(t) for t in self.tokens]
        for b in reqs:
            n, toks = len(new[b]), self.tokens[b]
            rows = [np.stack([p[table[b, s // 64], :, s % 64] for s in range(len(toks))]) for p in kv]
            x = self.qkv[layer][[t for t, _ in toks]].double().cpu().numpy()
            want = OC.qk_norm_rope(x[:, H:H + K], self.norm[1].double().cpu().numpy(), 1e-6, [p for _, p in toks],
                                   self.inv, D - R, False)
            eps = {"f32": 2.0 ** -16, "bf16": 2.0 ** -8, "fp8x132": 2.0 ** -4}[self.kind]
            top = np.abs(want).max(-1, keepdims=True)
            assert np.all(np.abs(rows[0] - want) <= eps * np.abs(want) * 1.01 + top * (2.0 ** -16 + (eps == 2.0 ** -4) * 2.0 ** -18))
            see = OC.window_rows(n, len(toks), window, sink) if bits is None else \
                OC.tree_rows(bits[b], len(toks), window, sink)
            ref = OC.attend(q[at:at + n].double().cpu().numpy(), rows[0], rows[1], see, SCALE)
            c = type("C", (), dict(kind=self.kind, head_dim=D))
            U.check_attend(f"request {b}", c, (out, lse), ref, at)
            at += n


@pytest.mark.parametrize("kind", ["bf16", "fp8x132", "f32"])
def test_serving_step(kind):
    s = Server(kind)
    rng = np.random.default_rng(4)
    ids = iter(rng.permutation(1000))
    take = lambda n, p0: [(int(next(ids)), p0 + i) for i in range(n)]  # noqa: E731
    # two prompts of unlike lengths, one past a page
    s.step({0: take(130, 0), 2: take(50, 0)}, window=100, sink=4)
    # a token each, with the window
    s.step({0: take(1, 130), 2: take(1, 50)}, window=100, sink=4)
    # a tree of drafts each: positions by depth
    new, bits = {}, {}
    for b, n in ((0, 12), (2, 20)):
        bits[b] = U.tree_bits(rng, n)
        base = len(s.tokens[b])
        new[b] = [(int(next(ids)), base + int(bits[b][i].sum()) - 1) for i in range(n)]
    s.step(new, bits=bits)
    # the deepest path of each is accepted, the rest goes
    start = {b: len(s.tokens[b]) - len(new[b]) for b in new}
    path = {b: np.flatnonzero(bits[b][int(bits[b].sum(1).argmax())]) for b in new}
    keep = torch.full((2, 32), -1, dtype=torch.int32)
    for i, b in enumerate((0, 2)):
        keep[i, :len(path[b])] = torch.from_numpy(path[b] + start[b]).to(torch.int32)
        s.tokens[b] = s.tokens[b][:start[b]] + [new[b][j] for j in path[b]]
    s.page("fm_cache_compact", s.ints([0, 2]), s.ints([start[0], start[2]]), keep.to(DEV), 32,
           s.ints([len(path[0]), len(path[2])]), 2)
    # request 0 is forked, shared and deep; each goes on by itself
    s.page("fm_cache_fork", s.ints([0]), s.ints([1]), 1, False)
    s.page("fm_cache_fork", s.ints([0]), s.ints([3]), 1, True)
    s.tokens[1], s.tokens[3] = list(s.tokens[0]), list(s.tokens[0])
    s.step({b: take(3, len(s.tokens[b])) for b in range(4)}, window=90, sink=2)
    # rejected tokens are cut, inside a page; another step
    cut = [len(s.tokens[b]) - 2 for b in (0, 1)]
    s.page("fm_cache_free", s.ints([0, 1]), s.ints(cut), 2)
    for b, n in zip((0, 1), cut):
        s.tokens[b] = s.tokens[b][:n]
    s.step({b: take(70, len(s.tokens[b])) for b in (0, 1)})
    # the end: every page is free again
    s.page("fm_cache_free", s.ints([0, 1, 2, 3]), None, 4)
    assert int(s.n_free) == 40 and not s.ref.any() and not s.lens.any()
    assert sorted(s.free.tolist()) == list(range(40)) and bool((s.table == -1).all())
