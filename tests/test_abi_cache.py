"""Host checks of the paged-cache entry points that need no GPU: every refusal comes before any
HIP call (the addresses are fake), and the ctypes descriptors match the header's structs."""
import ctypes as C
import os
import subprocess

import pytest

from tests.test_abi import FAKE, good_kv, status_of
from top_selection_fm_amd import api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = api.FM_ERR_INVALID_ARG, api.FM_ERR_UNSUPPORTED, api.FM_ERR_WORKSPACE


def layout(tmp_path, structs):
    lines = []
    for cname, cls in structs.items():
        lines.append(f'printf("{cname} sizeof %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f[0]} %zu\\n", offsetof({cname}, {f[0]}));' for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"fm.h\"\nint main(void) {\n"
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    return {tuple(x.split()[:2]): int(x.split()[2]) for x in out.splitlines()}


def check_layout(tmp_path, structs):
    got = layout(tmp_path, structs)
    for cname, cls in structs.items():
        assert got[(cname, "sizeof")] == C.sizeof(cls), cname
        for f in cls._fields_:
            assert got[(cname, f[0])] == getattr(cls, f[0]).offset, (cname, f[0])


# ------------------------------------------------------------------------------ attention
def good_attn(**kw):
    d = api.AttnDesc(FAKE, api.FM_BF16, 8 * 128, FAKE, 8 * 128, FAKE, FAKE, 2, 1, 8, 2, 0.1, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def attend_status(a, kv, window=100, n_sink=0, ws=None, nb=0):
    return status_of(api.fm_attend_window, a, kv, window, n_sink, ws, nb, 0)[0]


def test_attn_desc_layout(tmp_path):
    check_layout(tmp_path, {"fm_attn_desc": api.AttnDesc, "fm_kv_desc": api.KvDesc})


@pytest.mark.parametrize("kw,status", [
    (dict(q_dtype=api.FM_F32), UNSUPPORTED), (dict(q_dtype=api.FM_FP8_E4M3), UNSUPPORTED),
    (dict(T=-1), INVALID), (dict(max_rows=-1), INVALID), (dict(n_heads=9), INVALID), (dict(n_heads=0), INVALID),
    (dict(n_kv_heads=0), INVALID), (dict(n_heads=1026, q_ld=1026 * 128, out_ld=1026 * 128), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q_ld=1016), INVALID), (dict(out_ld=1016), INVALID),
    (dict(q_ld=1028), INVALID), (dict(out_ld=1028), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(q_start=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 8), INVALID),
    (dict(lse=FAKE + 2), INVALID), (dict(layer=-1), INVALID), (dict(layer=1), INVALID), (dict(layer=16), INVALID),
    (dict(max_rows=1 << 28, T=1 << 28), UNSUPPORTED),
])
def test_attend_refusals(kw, status):
    kv = good_kv(n_pools=2)
    assert attend_status(good_attn(**kw), kv) == status
    assert api.fm_attend_workspace_bytes(good_attn(**kw), kv, 100, 0) == 0
    mask = status_of(api.fm_attend_tree, good_attn(**kw), kv, FAKE, 1 << 24, 100, 0, None, 0, 0)
    assert mask[0] == status


def test_attend_refuses_caches():
    kv = good_kv(n_pools=2)
    assert attend_status(good_attn(), kv, window=0) == INVALID
    assert attend_status(good_attn(), kv, n_sink=-1) == INVALID
    assert attend_status(good_attn(), good_kv(n_pools=1)) == INVALID
    for field, value, status in (("head_dim", 96, UNSUPPORTED), ("page_size", 32, UNSUPPORTED), ("B", 0, INVALID),
                                 ("key_dtype", api.FM_FP8_E4M3, UNSUPPORTED), ("block_table", None, INVALID),
                                 ("n_phys_pages", 0, INVALID), ("bt_ld", 3, INVALID)):
        kv = good_kv(n_pools=2)
        setattr(kv, field, value)
        assert attend_status(good_attn(), kv) == status, field
    kv = good_kv("fp8x132", n_pools=2)
    kv.head_dim = 64
    assert attend_status(good_attn(), kv) == UNSUPPORTED


def test_attend_workspace():
    kv = good_kv(n_pools=2, max_seq_len=100000)
    need = api.fm_attend_workspace_bytes(good_attn(), kv, 1 << 40, 0)
    assert need > 0
    assert attend_status(good_attn(), kv, 1 << 40, 0, None, need) == WORKSPACE
    assert attend_status(good_attn(), kv, 1 << 40, 0, FAKE, need - 1) == WORKSPACE
    assert attend_status(good_attn(), kv, 1 << 40, 0, FAKE + 16, need) == WORKSPACE
    assert api.fm_attend_workspace_bytes(good_attn(), kv, 64, 0) == 0        # a page's window: one part


def test_attend_launch_limits():
    """More workgroups than a launch holds are refused; so many requests or rows that the joining
    launch cannot number them are taken whole."""
    kv = good_kv(n_pools=2, max_seq_len=100000)
    kv.B = 1 << 20
    assert attend_status(good_attn(), kv) == UNSUPPORTED
    kv.B = 70000
    assert api.fm_attend_workspace_bytes(good_attn(), kv, 1 << 40, 0) == 0
    kv.B = 1
    assert api.fm_attend_workspace_bytes(good_attn(max_rows=1 << 22, T=1 << 22), kv, 1 << 40, 0) == 0


def test_attend_tree_refusals():
    kv, a = good_kv(n_pools=2), good_attn(max_rows=65, T=65)
    st = lambda mask, ld: status_of(api.fm_attend_tree, a, kv, mask, ld, 100, 0, None, 0, 0)[0]  # noqa: E731
    assert st(FAKE, 0) == INVALID and st(FAKE, 1) == INVALID
    assert st(None, 2) == INVALID and st(FAKE + 4, 2) == INVALID


def test_attend_zero_rows_is_a_noop():
    kv = good_kv(n_pools=2)
    api.fm_attend_window(good_attn(T=0, q=None, out=None, q_start=None), kv, 100, 0, None, 0, 0)
    api.fm_attend_window(good_attn(max_rows=0), kv, 100, 0, None, 0, 0)
    api.fm_attend_tree(good_attn(T=0), kv, None, 1, 100, 0, None, 0, 0)
    assert api.fm_last_error() == ""


# ------------------------------------------------------------------------------ norms and rotation
def good_qk(**kw):
    d = api.QkDesc(FAKE, FAKE, FAKE, 8 * 128, 256, 256, FAKE, None, 8 * 128, 0, FAKE, FAKE, api.FM_BF16, 2, 8, 2, 128,
                   FAKE, None, None, 0, 1e-6, 64, 64, 0, 160000.0, 16.0, 65536, 32.0, 1.0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_qk_desc_layout(tmp_path):
    check_layout(tmp_path, {"fm_qk_desc": api.QkDesc, "fm_cache_desc": api.CacheDesc})


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=api.FM_FP8_E4M3), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(T=-1), INVALID),
    (dict(T=(1 << 22) + 1), INVALID), (dict(n_heads=-1), INVALID), (dict(n_heads=0, n_kv_heads=0), INVALID),
    (dict(n_heads=1025), UNSUPPORTED), (dict(rms_eps=-1.0), INVALID), (dict(rms_eps=float("nan")), INVALID),
    (dict(rope_dim=63), INVALID), (dict(rope_first=63), INVALID), (dict(rope_first=66), INVALID),
    (dict(rope_dim=-2), INVALID), (dict(rope_first=-2), INVALID), (dict(rope_first=130, rope_dim=0), INVALID),
    (dict(rope_halves=2), INVALID), (dict(rope_halves=1, rope_dim=8), UNSUPPORTED),
    (dict(rope_halves=1, rope_first=4, rope_dim=32), UNSUPPORTED), (dict(rope_base=1.0), INVALID),
    (dict(rope_factor=0.5), INVALID), (dict(rope_orig_len=0), INVALID), (dict(beta_fast=0.5), INVALID),
    (dict(beta_slow=0.0), INVALID), (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(q_ld=1016), INVALID),
    (dict(q_ld=1028), INVALID), (dict(q_out=None), INVALID), (dict(q_out_ld=1016), INVALID), (dict(k=None), INVALID),
    (dict(k_ld=248), INVALID), (dict(v=None), INVALID), (dict(v_ld=255), INVALID), (dict(k_out=FAKE + 4), INVALID),
    (dict(k_out=FAKE, k_out_ld=256 + 4), INVALID), (dict(q_norm=FAKE + 2), INVALID), (dict(k_norm=FAKE + 8), INVALID),
    (dict(pos=None), INVALID), (dict(layer=1), INVALID), (dict(T=3), INVALID), (dict(n_kv_heads=0), INVALID),
    (dict(q_out_ld=2048), INVALID),                                     # in place with another ld
])
def test_qk_refusals(kw, status):
    assert status_of(api.fm_qk_norm_rope, good_qk(**kw), good_kv(n_pools=2), 0)[0] == status


def test_qk_refuses_caches():
    st = lambda d, kv: status_of(api.fm_qk_norm_rope, d, kv, 0)[0]  # noqa: E731
    assert st(good_qk(), good_kv("f32", n_pools=2)) == UNSUPPORTED
    assert st(good_qk(dtype=api.FM_F32), good_kv("bf16", n_pools=2)) == UNSUPPORTED
    assert st(good_qk(head_dim=64, rope_first=0), good_kv(n_pools=2)) == INVALID
    assert st(good_qk(), None) == INVALID                               # nowhere for the keys
    assert st(good_qk(), good_kv(n_pools=1)) == INVALID
    api.fm_qk_norm_rope(good_qk(T=0, q=None, pos=None), good_kv(n_pools=2), 0)
    assert api.fm_last_error() == ""


# ------------------------------------------------------------------------------ pages
def good_cache(**kw):
    d = api.CacheDesc()
    d.pool[0], d.heads[0], d.row_bytes[0], d.n_pools = FAKE, 2, 256, 1
    d.block_table = d.seq_lens = d.ref = d.free_list = d.n_free = FAKE
    d.bt_ld, d.B, d.n_phys_pages = 10, 4, 100
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def cache_calls(c, n=2, ws=FAKE, nb=1 << 20, lists=FAKE):
    return [status_of(f, *a)[0] for f, a in (
        (api.fm_cache_fork, (c, lists, FAKE, n, False, None, ws, nb, 0)),
        (api.fm_cache_grow, (c, lists, FAKE, n, None, ws, nb, 0)),
        (api.fm_cache_free, (c, lists, None, n, None, 0)),
        (api.fm_cache_compact, (c, lists, FAKE, FAKE, 4, FAKE, n, None, 0)))]


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(B=16385), UNSUPPORTED), (dict(bt_ld=0), INVALID), (dict(bt_ld=1 << 30), INVALID),
    (dict(n_phys_pages=0), INVALID), (dict(n_phys_pages=(1 << 19) + 1), UNSUPPORTED), (dict(n_pools=0), INVALID),
    (dict(n_pools=33), INVALID), (dict(n_pools=2), INVALID), (dict(block_table=None), INVALID), (dict(ref=None), INVALID),
    (dict(seq_lens=None), INVALID), (dict(free_list=None), INVALID), (dict(n_free=None), INVALID),
])
def test_cache_refusals(kw, status):
    c = good_cache(**kw)
    assert cache_calls(c) == [status] * 4
    assert api.fm_cache_workspace_bytes(c, 2) == 0


def test_cache_pool_shapes():
    for field, value in (("row_bytes", 6), ("row_bytes", 0), ("row_bytes", 1 << 17), ("heads", 0), ("heads", 1025)):
        c = good_cache()
        getattr(c, field)[0] = value
        assert cache_calls(c) == [INVALID] * 4, field
    c = good_cache()
    c.pool[0] = FAKE + 4
    assert cache_calls(c) == [INVALID] * 4


def test_cache_entries_and_workspace():
    c = good_cache()
    assert cache_calls(c, n=-1) == [INVALID] * 4
    assert cache_calls(c, n=16385) == [UNSUPPORTED] * 4
    assert cache_calls(c, lists=None) == [INVALID] * 4
    need = api.fm_cache_workspace_bytes(c, 100)
    assert need >= 1600
    for ws, nb in ((None, need), (FAKE + 16, need), (FAKE, need - 1)):
        assert status_of(api.fm_cache_fork, c, FAKE, FAKE, 100, False, None, ws, nb, 0)[0] == WORKSPACE
        assert status_of(api.fm_cache_grow, c, FAKE, FAKE, 100, None, ws, nb, 0)[0] == WORKSPACE
    assert status_of(api.fm_cache_compact, c, FAKE, FAKE, FAKE, -1, FAKE, 2, None, 0)[0] == INVALID
    assert status_of(api.fm_cache_compact, c, FAKE, FAKE, None, 4, FAKE, 2, None, 0)[0] == INVALID
    for call in (lambda: api.fm_cache_fork(c, None, None, 0), lambda: api.fm_cache_grow(c, None, None, 0),
                 lambda: api.fm_cache_free(c, None, None, 0), lambda: api.fm_cache_compact(c, None, None, None, 0, None, 0)):
        call()
        assert api.fm_last_error() == ""
