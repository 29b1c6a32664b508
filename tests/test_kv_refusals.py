"""What the BF16 paged cache's calls refuse before they touch a device, the
structs' layout, and the rotary frequencies (no GPU)."""
from __future__ import annotations

import ctypes as C
import math

import pytest

from persistent_moe_decode_gb300 import build as B
from persistent_moe_decode_gb300 import kv, mk


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mk.lib()


P = 1 << 20     # an aligned address that no refused call reads
R, BF, F32 = mk.mk_head_rows, mk.MK_TYPE_BF16, mk.MK_TYPE_F32


def cache(**kw):
    f = dict(k_pool=P, v_pool=2 * P, num_pages=4, n_kv_heads=2, head_dim=64, status=None)
    f.update(kw)
    return mk.mk_kv_cache(**f)


def rope(**kw):
    f = dict(turns=P, head_dim=64, rotary_dim=32, interleaved=0, magnitude=1.0)
    f.update(kw)
    return mk.mk_rope(**f)


def test_struct_layout_matches_header(lib, tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    structs = (mk.mk_kv_cache, mk.mk_rope, mk.mk_head_rows)
    lines = []
    for st in structs:
        lines.append(f'printf("{st.__name__} %zu\\n", sizeof({st.__name__}));')
        for name, _ in st._fields_:
            lines.append(f'printf("{st.__name__}.{name} %zu\\n", offsetof({st.__name__}, {name}));')
    (tmp_path / "l.c").write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mk.h"\nint main(void) {\n'
                                  + "\n".join(lines) + "\nreturn 0;\n}\n")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")],
                   check=True)
    out = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split("\n")
    got = dict(line.split() for line in out if line)
    for st in structs:
        assert int(got[st.__name__]) == C.sizeof(st)
        for name, _ in st._fields_:
            assert int(got[f"{st.__name__}.{name}"]) == getattr(st, name).offset


BAD_CACHE = [(dict(head_dim=96), mk.MK_ERR_BAD_CONFIG), (dict(n_kv_heads=0), mk.MK_ERR_BAD_CONFIG),
             (dict(n_kv_heads=1025), mk.MK_ERR_BAD_CONFIG), (dict(num_pages=0), mk.MK_ERR_BAD_CONFIG),
             (dict(num_pages=1 << 26), mk.MK_ERR_BAD_CONFIG), (dict(k_pool=None), mk.MK_ERR_BAD_ARG),
             (dict(v_pool=None), mk.MK_ERR_BAD_ARG), (dict(v_pool=P + 8), mk.MK_ERR_BAD_ARG),
             (dict(status=P + 2), mk.MK_ERR_BAD_ARG)]
BAD_ROPE = [(dict(turns=None), mk.MK_ERR_BAD_ARG), (dict(turns=P + 4), mk.MK_ERR_BAD_ARG),
            (dict(head_dim=80), mk.MK_ERR_BAD_CONFIG), (dict(rotary_dim=0), mk.MK_ERR_BAD_CONFIG),
            (dict(rotary_dim=8), mk.MK_ERR_BAD_CONFIG), (dict(rotary_dim=24), mk.MK_ERR_BAD_CONFIG),
            (dict(rotary_dim=80), mk.MK_ERR_BAD_CONFIG), (dict(interleaved=2), mk.MK_ERR_BAD_CONFIG),
            (dict(magnitude=math.nan), mk.MK_ERR_BAD_ARG), (dict(magnitude=math.inf), mk.MK_ERR_BAD_ARG)]


def refused(fn, code, *args):
    with pytest.raises(mk.MkError) as e:
        fn(*args)
    assert e.value.code == code


def apply_args(**kw):
    f = dict(rope=rope(), n=3, positions=P, type=BF, q=R(P, 4, 256, 64), k=R(P, 2, 128, 64), q_out=R(P, 4, 256, 64),
             k_out=R(P, 2, 128, 64))
    f.update(kw)
    return list(f.values())


@pytest.mark.parametrize("bad,code", BAD_ROPE)
def test_bad_rope(lib, bad, code):
    refused(mk.mk_rope_apply, code, *apply_args(rope=rope(**bad)))


@pytest.mark.parametrize("bad,code", [
    (dict(n=-1), mk.MK_ERR_BAD_ARG), (dict(positions=None), mk.MK_ERR_BAD_ARG), (dict(positions=P + 2), mk.MK_ERR_BAD_ARG),
    (dict(type=7), mk.MK_ERR_BAD_ARG), (dict(q=R(None, 4, 256, 64)), mk.MK_ERR_BAD_ARG),
    (dict(q=R(P + 8, 4, 256, 64)), mk.MK_ERR_BAD_ARG), (dict(q=R(P, 4, 260, 64)), mk.MK_ERR_BAD_ARG),
    (dict(k=R(P, 2, 128, 68)), mk.MK_ERR_BAD_ARG), (dict(q_out=R(P, 3, 256, 64)), mk.MK_ERR_BAD_ARG),
    (dict(q=R(P, -1, 256, 64)), mk.MK_ERR_BAD_CONFIG), (dict(k=R(P, 65537, 256, 64)), mk.MK_ERR_BAD_CONFIG),
    # outputs whose rows or heads overlap
    (dict(q_out=R(P, 4, 192, 64)), mk.MK_ERR_BAD_ARG), (dict(q_out=R(P, 4, 256, 32)), mk.MK_ERR_BAD_ARG),
    (dict(k_out=R(P, 2, 0, 64)), mk.MK_ERR_BAD_ARG), (dict(k_out=R(P, 2, 64, 128)), mk.MK_ERR_BAD_ARG),
    (dict(k_out=R(P, 2, -128, 64)), mk.MK_ERR_BAD_ARG)])
def test_bad_rotary_call(lib, bad, code):
    refused(mk.mk_rope_apply, code, *apply_args(**bad))


def append_args(**kw):
    f = dict(cache=cache(), rope=rope(), n=3, positions=P, type=BF, q=R(P, 4, 256, 64), k=R(P, 2, 128, 64),
             v=R(P, 2, 128, 64), slots=P, q_out=R(P, 4, 256, 64))
    f.update(kw)
    return list(f.values())


@pytest.mark.parametrize("bad,code", BAD_CACHE)
def test_bad_cache(lib, bad, code):
    c = cache(**bad)
    refused(mk.mk_kv_append, code, *append_args(cache=c))
    refused(mk.mk_kv_attention, code, *attn_args(cache=c))
    assert mk.mk_kv_workspace(c, 4, 10, 2, 0) == 0


@pytest.mark.parametrize("bad,code", [
    (dict(rope=rope(head_dim=128)), mk.MK_ERR_BAD_CONFIG), (dict(slots=None), mk.MK_ERR_BAD_ARG),
    (dict(slots=P + 1), mk.MK_ERR_BAD_ARG), (dict(positions=None), mk.MK_ERR_BAD_ARG),
    (dict(k=R(P, 3, 192, 64)), mk.MK_ERR_BAD_ARG), (dict(v=R(P, 1, 128, 64)), mk.MK_ERR_BAD_ARG),
    (dict(type=F32, v=R(P, 2, 126, 64)), mk.MK_ERR_BAD_ARG), (dict(n=-4), mk.MK_ERR_BAD_ARG),
    (dict(q_out=R(P, 4, 128, 64)), mk.MK_ERR_BAD_ARG)])
def test_bad_append(lib, bad, code):
    refused(mk.mk_kv_append, code, *append_args(**bad))


def attn_args(**kw):
    f = dict(cache=cache(), q=P, q_stride=256, out=P, out_stride=256, hq=4, total_q=10, batch=2, q_starts=P, tables=P,
             max_pages=4, lens=P, groups=0, group_starts=None, prefix_lens=None, scale=0.1, ws=None, ws_bytes=0)
    f.update(kw)
    return list(f.values())


@pytest.mark.parametrize("bad,code", [
    (dict(hq=3), mk.MK_ERR_BAD_CONFIG), (dict(hq=0), mk.MK_ERR_BAD_CONFIG), (dict(hq=258), mk.MK_ERR_BAD_CONFIG),
    (dict(total_q=-1), mk.MK_ERR_BATCH_TOO_LARGE), (dict(total_q=(1 << 24) + 1), mk.MK_ERR_BATCH_TOO_LARGE),
    (dict(batch=-1), mk.MK_ERR_BATCH_TOO_LARGE), (dict(batch=65536), mk.MK_ERR_BATCH_TOO_LARGE),
    (dict(groups=-1), mk.MK_ERR_BATCH_TOO_LARGE), (dict(groups=65536), mk.MK_ERR_BATCH_TOO_LARGE),
    (dict(max_pages=-1), mk.MK_ERR_BAD_ARG), (dict(max_pages=1 << 26), mk.MK_ERR_BAD_ARG),
    (dict(max_pages=(1 << 24) + 1), mk.MK_ERR_BAD_ARG),     # above it one item could outlast the kernel's waits
    (dict(scale=0.0), mk.MK_ERR_BAD_ARG), (dict(scale=-1.0), mk.MK_ERR_BAD_ARG), (dict(scale=math.nan), mk.MK_ERR_BAD_ARG),
    (dict(scale=math.inf), mk.MK_ERR_BAD_ARG), (dict(scale=2.0 ** 20), mk.MK_ERR_BAD_ARG),
    (dict(q=None), mk.MK_ERR_BAD_ARG), (dict(out=None), mk.MK_ERR_BAD_ARG), (dict(q=P + 8), mk.MK_ERR_BAD_ARG),
    (dict(out=P + 4), mk.MK_ERR_BAD_ARG), (dict(q_stride=260), mk.MK_ERR_BAD_ARG), (dict(out_stride=252), mk.MK_ERR_BAD_ARG),
    (dict(q_stride=128), mk.MK_ERR_BAD_ARG), (dict(out_stride=248), mk.MK_ERR_BAD_ARG),
    (dict(q_starts=None), mk.MK_ERR_BAD_ARG), (dict(tables=None), mk.MK_ERR_BAD_ARG), (dict(lens=None), mk.MK_ERR_BAD_ARG),
    (dict(groups=1), mk.MK_ERR_BAD_ARG), (dict(groups=1, group_starts=P), mk.MK_ERR_BAD_ARG)])
def test_bad_attention(lib, bad, code):
    refused(mk.mk_kv_attention, code, *attn_args(**bad))


def test_nothing_to_do_touches_no_device(lib):
    assert mk.mk_rope_apply(*apply_args(n=0, positions=None)) == 0
    assert mk.mk_kv_append(*append_args(n=0, positions=None, slots=None)) == 0
    assert mk.mk_kv_attention(*attn_args(total_q=0)) == 0
    assert mk.mk_kv_attention(*attn_args(batch=0)) == 0
    none = R(None, 0, 0, 0)
    assert mk.mk_rope_apply(*apply_args(q=none, q_out=none, k=none, k_out=none)) == 0


def test_null_structs(lib):
    L = lib
    assert L.mk_kv_attention(None, *attn_args()[1:], None) == mk.MK_ERR_BAD_ARG
    a = append_args()
    assert L.mk_kv_append(None, *a[1:], None) == mk.MK_ERR_BAD_ARG
    for i in (1, 5, 6, 7, 9):
        assert L.mk_kv_append(*[None if j == i else x for j, x in enumerate(a)], None) == mk.MK_ERR_BAD_ARG, i
    a = apply_args()
    for i in (0, 4, 5, 6, 7):
        assert L.mk_rope_apply(*[None if j == i else x for j, x in enumerate(a)], None) == mk.MK_ERR_BAD_ARG, i


def test_frequencies():
    f, m = kv.frequencies(64, 1e4)
    assert m == 1 and f[0] == 1 and abs(f[31] - 1e4 ** (-62 / 64)) < 1e-18
    g, m = kv.frequencies(64, 1e4, "linear", 4.0)
    assert m == 1 and (g == f / 4).all()
    g, m = kv.frequencies(64, 1e4, "ntk", 4.0)
    assert m == 1 and g[0] == 1 and abs(g[31] * 4 / f[31] - 1) < 1e-12      # the slowest pair is slowed by the factor
    g, m = kv.frequencies(64, 1e4, "yarn", 4.0, original_context=4096)
    assert abs(m - (1 + 0.1 * math.log(4))) < 1e-15 and g[0] == f[0] and g[31] == f[31] / 4
    assert all(a >= b for a, b in zip(f, g))
    for bad in (dict(theta=1.0), dict(theta=math.nan), dict(theta=1e4, scaling="other"),
                dict(theta=1e4, scaling="linear", factor=0.5), dict(theta=1e4, scaling="yarn", factor=2.0),
                dict(theta=1e4, scaling="yarn", factor=2.0, original_context=64, beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(ValueError):
            kv.frequencies(64, **bad)


def test_python_refusals_without_a_gpu():
    import torch
    for kw in (dict(head_dim=96), dict(head_dim=64, rotary_dim=24), dict(head_dim=64, rotary_dim=80),
               dict(head_dim=64, rotary_dim=0)):
        with pytest.raises(ValueError):
            kv.Rope(theta=1e4, device="cpu", **kw)
    with pytest.raises(ValueError, match="GPU"):
        kv.Rope(64, 1e4, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        kv.PagedCache(4, 2, 64, device="cpu")
    z = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    for k, v in ((z.float(), z), (z, z[:3]), (z[0], z[0]), (z[:, :, :8], z[:, :, :8]), (z[:0], z[:0])):
        with pytest.raises(ValueError):
            kv.PagedCache.from_pools(k, v)
