"""The paged-cache calls on pages whose bytes lie past 2^32: the same bits as on a small pool."""
from __future__ import annotations

import pytest
import torch

from tests import cache_util as U
from top_selection_fm_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
K, H, D, SMALL, WIDTH = 8, 16, 128, 40, 10


def run(kind, pages, shift):
    """Grow, write, fork, compact and attend on pages shift .. shift + SMALL - 1 of `pages`."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    row, dt = {"bf16": (D, torch.bfloat16), "fp8x132": (132, torch.uint8), "f32": (D, torch.float32)}[kind]
    pools = [torch.empty(pages, K, 64, row, dtype=dt, device=DEV) for _ in range(2)]
    for p in pools:
        p[shift:shift + SMALL] = 0
    table, lens = torch.full((3, WIDTH), -1, dtype=torch.int32, device=DEV), i32([0, 0, 0])
    ref, free, n_free = torch.zeros(pages, dtype=torch.int32, device=DEV), i32(range(pages)), i32([shift + SMALL])
    c = api.cache_desc(pools, table, lens, ref, free, n_free)
    kv = api.kv_desc(pools, kind, table, lens, 64 * WIDTH)
    ws = torch.empty(api.fm_cache_workspace_bytes(c, 2), dtype=torch.uint8, device=DEV)
    ok = torch.zeros(4, dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(1)
    T = 460
    qdt = U.TORCH[kind]
    qkv = torch.randn(T, H + 2 * K, D, generator=g).to(qdt).to(DEV)
    w = torch.ones(D, dtype=qdt, device=DEV)
    api.fm_cache_grow(c, i32([0, 1]), i32([300, 160]), 2, ok=ok, ws=ws, ws_bytes=ws.numel())
    req, slot = i32([0] * 300 + [1] * 160), i32(list(range(300)) + list(range(160)))
    name = "f32" if kind == "f32" else "bf16"
    api.fm_qk_norm_rope(api.qk_desc(qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:], name, qkv[:, :H], w, w, slot,
                                    row_req=req, slot=slot, rope_dim=64), kv)
    api.fm_cache_fork(c, i32([1]), i32([2]), 1, True, ok=ok[2:], ws=ws, ws_bytes=ws.numel())
    api.fm_cache_compact(c, i32([0]), i32([100]), i32([list(range(101, 300, 2))]), 100, i32([100]), 1, ok=ok[3:])
    outs = []
    for rows in ([1, 1, 1], [60, 50, 70]):
        q = qkv[:sum(rows), :H].contiguous()
        start = i32([0, rows[0], rows[0] + rows[1], sum(rows)])
        out, lse = torch.empty_like(q), torch.empty(sum(rows), H, device=DEV)
        d = api.attn_desc(q, name, out, start, max(rows), n_kv_heads=K, scale=0.1, lse=lse)
        nb = api.fm_attend_workspace_bytes(d, kv, 1 << 20, 0)
        aws = torch.empty(max(nb, 256), dtype=torch.uint8, device=DEV)
        api.fm_attend_window(d, kv, 1 << 20, 0, aws, nb)
        outs += [out, lse]
    torch.cuda.synchronize()
    assert ok.tolist() == [1, 1, 1, 1] and lens.tolist() == [200, 160, 160]
    used = table[table >= 0]
    assert int(used.min()) >= shift
    moved = [p[shift:shift + SMALL].clone().view(torch.uint8) for p in pools]
    return outs + moved + [torch.where(table < 0, table, table - shift), ref[shift:shift + SMALL]]


@pytest.mark.parametrize("kind", ["bf16", "fp8x132", "f32"])
def test_pages_past_four_gibibytes(kind):
    page = K * 64 * {"bf16": 256, "fp8x132": 132, "f32": 512}[kind]
    pages = (1 << 32) // page + 500
    assert (pages - SMALL) * page > 1 << 32
    near, far = run(kind, SMALL, 0), run(kind, pages, pages - SMALL)
    for i, (a, b) in enumerate(zip(near, far)):
        assert torch.equal(a, b), i
        assert i > 3 or bool(torch.isfinite(a.float()).all())
