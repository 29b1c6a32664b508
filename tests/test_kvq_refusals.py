"""What the 4-bit cache's calls refuse before they touch a device (no GPU), and
the format's restatement against its own promises."""
from __future__ import annotations

import ctypes as C

import numpy as np
import pytest
import torch

from persistent_moe_decode_gb300 import build as B
from persistent_moe_decode_gb300 import kvq, mk
from tests import _kvq


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mk.lib()


P = 1 << 20     # an aligned address that no refused call reads


def cache(**kw):
    f = dict(pool=P, num_pages=4, n_kv_heads=2, head_dim=64, status=None)
    f.update(kw)
    return mk.mk_kvq_cache(**f)


def rows(**kw):
    f = dict(k=P, v=P, type=mk.MK_TYPE_BF16, count=8, page_stride=2048, row_stride=128, head_stride=64)
    f.update(kw)
    return mk.mk_kv_rows(**f)


def test_page_bytes(lib):
    assert mk.mk_kvq_page_bytes(4, 128) == 4 * 2304 and mk.mk_kvq_page_bytes(2, 64) == 2 * 1152
    for hkv, d in ((0, 64), (-1, 128), (4, 96), (4, 0), (4, 256)):
        assert mk.mk_kvq_page_bytes(hkv, d) == 0
        with pytest.raises(ValueError):
            kvq.page_bytes(hkv, d)


def test_struct_layout_matches_header(lib, tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lines = []
    for st in (mk.mk_kvq_cache, mk.mk_kv_rows):
        lines.append(f'printf("{st.__name__} %zu\\n", sizeof({st.__name__}));')
        for name, _ in st._fields_:
            lines.append(f'printf("{st.__name__}.{name} %zu\\n", offsetof({st.__name__}, {name}));')
    (tmp_path / "l.c").write_text('#include <stdio.h>\n#include <stddef.h>\n#include "mk.h"\nint main(void) {\n'
                                  + "\n".join(lines) + "\nreturn 0;\n}\n")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")],
                   check=True)
    out = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split("\n")
    got = dict(line.split() for line in out if line)
    for st in (mk.mk_kvq_cache, mk.mk_kv_rows):
        assert int(got[st.__name__]) == C.sizeof(st)
        for name, _ in st._fields_:
            assert int(got[f"{st.__name__}.{name}"]) == getattr(st, name).offset


@pytest.mark.parametrize("bad,code", [
    (dict(head_dim=96), mk.MK_ERR_BAD_CONFIG), (dict(n_kv_heads=0), mk.MK_ERR_BAD_CONFIG),
    (dict(n_kv_heads=1025), mk.MK_ERR_BAD_CONFIG), (dict(num_pages=0), mk.MK_ERR_BAD_CONFIG),
    (dict(num_pages=1 << 27), mk.MK_ERR_BAD_CONFIG), (dict(pool=None), mk.MK_ERR_BAD_ARG),
    (dict(pool=P + 8), mk.MK_ERR_BAD_ARG), (dict(status=P + 2), mk.MK_ERR_BAD_ARG)])
def test_bad_caches(lib, bad, code):
    c, r = cache(**bad), rows()
    assert lib.mk_kvq_write(C.byref(c), C.byref(r), P, P, 1, 1, None) == code
    assert lib.mk_kvq_read(C.byref(c), P, C.byref(r), P, 1, 1, None) == code
    assert lib.mk_kvq_attention(C.byref(c), P, 256, P, 256, 0, 4, 1, P, 4, P, 1.0, None, 0, None) == code
    assert mk.mk_kvq_workspace(c, 0, 4, 1, 4000) == 0


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(k=P + 8), dict(type=2), dict(count=-1),
                                 dict(row_stride=100), dict(page_stride=2044), dict(head_stride=63),
                                 dict(type=mk.MK_TYPE_F32, row_stride=126)])
def test_bad_rows(lib, bad):
    c, r = cache(), rows(**bad)
    assert lib.mk_kvq_write(C.byref(c), C.byref(r), P, P, 2, 1, None) == mk.MK_ERR_BAD_ARG
    assert lib.mk_kvq_read(C.byref(c), P, C.byref(r), P, 2, 1, None) == mk.MK_ERR_BAD_ARG


def test_bad_counts(lib):
    c, r = cache(), rows()
    for n, unit in ((-1, 1), (1, 2), (1, 0), (1 << 28, 16)):
        assert lib.mk_kvq_write(C.byref(c), C.byref(r), P, P, n, unit, None) == mk.MK_ERR_BAD_ARG
        assert lib.mk_kvq_read(C.byref(c), P, C.byref(r), P, n, unit, None) == mk.MK_ERR_BAD_ARG
    # implied indexes past the rows, past the cache
    assert lib.mk_kvq_write(C.byref(c), C.byref(r), None, P, 9, 1, None) == mk.MK_ERR_BAD_ARG
    assert lib.mk_kvq_write(C.byref(c), C.byref(rows(count=100)), None, None, 65, 1, None) == mk.MK_ERR_BAD_PAGE
    assert lib.mk_kvq_read(C.byref(c), None, C.byref(rows(count=100)), P, 5, 16, None) == mk.MK_ERR_BAD_PAGE
    assert lib.mk_kvq_write(None, C.byref(r), P, P, 1, 1, None) == mk.MK_ERR_BAD_ARG
    assert lib.mk_kvq_write(C.byref(c), None, P, P, 1, 1, None) == mk.MK_ERR_BAD_ARG
    # nothing to do
    assert lib.mk_kvq_write(C.byref(c), C.byref(rows(k=None, v=None, count=0)), None, None, 0, 1, None) == mk.MK_OK
    assert lib.mk_kvq_read(C.byref(c), None, C.byref(rows(k=None, v=None, count=0)), None, 0, 16, None) == mk.MK_OK


def test_bad_attention_arguments(lib):
    c = cache()

    def call(q=P, qs=256, out=P, os_=256, dtype=0, hq=4, batch=2, pt=P, mp=4, ln=P, scale=0.125, ws=P, wb=1 << 40):
        return lib.mk_kvq_attention(C.byref(c), q, qs, out, os_, dtype, hq, batch, pt, mp, ln, scale, ws, wb, None)

    for kw in (dict(q=None), dict(out=None), dict(ln=None), dict(pt=None), dict(q=P + 8), dict(out=P + 4),
               dict(qs=252), dict(os_=260 - 2), dict(os_=128), dict(dtype=2), dict(dtype=-1), dict(mp=-1),
               dict(mp=1 << 28), dict(scale=float("nan")), dict(scale=float("inf")), dict(dtype=1, qs=254)):
        assert call(**kw) == mk.MK_ERR_BAD_ARG, kw
    for hq in (0, 3, -4, 65538):
        assert call(hq=hq) == mk.MK_ERR_BAD_CONFIG
    for b in (-1, 65536):
        assert call(batch=b) == mk.MK_ERR_BATCH_TOO_LARGE
    assert call(batch=0, q=None, out=None, ln=None) == mk.MK_OK


def test_a_cache_is_on_a_gpu():
    pool = torch.zeros(3, 2 * 1152, dtype=torch.uint8)
    with pytest.raises(ValueError):
        kvq.QuantCache.from_pool(pool, 2, 64)
    with pytest.raises(ValueError):
        kvq.QuantCache.from_pool(pool[:, :100], 2, 64)
    with pytest.raises(ValueError):
        kvq.QuantCache.from_pool(pool.float(), 2, 64)


# --------------------------------------------- the restatement's own promises

@pytest.mark.parametrize("d", [64, 128])
def test_every_code_has_its_own_place(d):
    """The record's addresses are a bijection: no two elements share a nibble, none falls outside."""
    t, i = np.meshgrid(np.arange(16), np.arange(d), indexing="ij")
    seen = []
    for at in (_kvq.key_at, _kvq.value_at):
        byte, odd = at(d, t, i)
        seen.append((2 * byte + odd).ravel())
    assert np.array_equal(np.sort(np.concatenate(seen)), np.arange(32 * d))
    tg = [_kvq.scale_at(d, tt, g, v) for v in (False, True) for tt in range(16) for g in range(d // 64)]
    assert sorted(tg) == list(range(16 * d, 18 * d, 4))


@pytest.mark.parametrize("d", [64, 128])
def test_the_restated_store_and_load_agree_within_half_a_step(d):
    rng = np.random.default_rng(d)
    hkv, n = 2, 40
    pool = rng.integers(0, 256, size=(5, hkv * 18 * d), dtype=np.uint8)
    k, v = (rng.normal(size=(n, hkv, d)).astype(np.float32).astype(np.float64) for _ in range(2))
    slots = rng.permutation(80)[:n]
    _kvq.store(pool, hkv, d, k, v, slots)
    for x, (code, step, low) in zip((k, v), _kvq.load(pool, hkv, d, slots)):
        assert (np.abs(step * code + low - x) <= 0.5 * step * (1 + 1e-6)).all()
        g = x.reshape(n, hkv, -1, 64)
        span = g.max(-1) - g.min(-1)
        assert (step.reshape(n, hkv, -1, 64)[..., 0] <= (span + 2.0 ** -7 * np.abs(g.min(-1))) / 15 * (1 + 2.0 ** -7)).all()


def test_the_step_refuses_unknown_cache_formats_and_shapes(lib):
    from persistent_moe_decode_gb300.configs import TINY
    w = mk.mk_weights()
    for bad in (2, -1):
        cfg = mk.make_config(TINY, 1, 8, 16, kv_format=bad)
        h = C.c_void_p()
        assert lib.mk_create(C.byref(cfg), C.byref(w), C.byref(h)) == mk.MK_ERR_BAD_CONFIG

    class Model:
        dims, fp8 = TINY, None
        w_gate = w_up = w_down = None

    for pool in (torch.zeros(2, 4, 100, dtype=torch.uint8), torch.zeros(4, 2 * 1152, dtype=torch.uint8),
                 torch.zeros(2, 4, 2 * 1152)):
        with pytest.raises(ValueError):
            mk.Decoder(Model, pool, None, 1, 4)


def test_attention_sms_over_the_4_bit_cache(lib):
    """The measured best splits of 152 SMs on the 30B/3.3B shape; the BF16 cache's are what they were."""
    from persistent_moe_decode_gb300.configs import A3B
    for lens, bf16, int4 in (([8192], 40, 56), ([262144], 128, 128), ([8192] * 4, 24, 32), ([8192] * 16, 36, 36),
                             ([16384] * 16, 36, 52), ([30000] * 16, 36, 64)):
        for fmt, want in ((mk.MK_KV_BF16, bf16), (mk.MK_KV_INT4, int4)):
            cfg = mk.make_config(A3B, len(lens), 16400, 1 << 20, kv_format=fmt)
            assert mk.mk_plan_step(cfg, 152, len(lens), np.array(lens))["n_attn"] == want


def test_bytes_of_a_cached_token():
    """4.5 bits a value: the record's 18 bytes for every 32 values, keys and values together."""
    from persistent_moe_decode_gb300.configs import A3B, TINY, WORKLOADS, algorithmic_bytes
    for d in (TINY, A3B):
        page = mk.mk_kvq_page_bytes(d.n_kv_heads, d.head_dim)
        assert d.kv_bytes_per_token("int4") * 16 == d.n_layers * page
        assert d.kv_bytes_per_token() == d.n_layers * 4 * d.n_kv_heads * d.head_dim
        n = [d.top_k] * d.n_layers
        assert algorithmic_bytes(d, n, [100], kv_format="int4") - algorithmic_bytes(d, n, [99], kv_format="int4") \
            == d.kv_bytes_per_token("int4")
    assert WORKLOADS["a3b_256k_kv4"].kv_format == "int4"
