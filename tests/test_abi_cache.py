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
