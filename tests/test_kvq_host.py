"""The 4-bit cache's calls on the host alone (no GPU): where the device cannot
be asked, and the pools a Decoder refuses."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from persistent_moe_decode_gb300 import build as B
from persistent_moe_decode_gb300 import kvq, mk

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mk.lib()


NO_DEVICE = """
import ctypes as C
from persistent_moe_decode_gb300 import mk
L, P = mk.lib(), 1 << 20
for d in (64, 128):
    for kind in (mk.MK_TYPE_BF16, mk.MK_TYPE_F32):
        c = mk.mk_kvq_cache(pool=P, num_pages=64, n_kv_heads=4, head_dim=d, status=None)
        r = mk.mk_kv_rows(P, 2 * P, kind, 16, 64 * d, d, 16 * d)
        for unit in (1, 16):
            assert L.mk_kvq_write(c, r, P, P, 3, unit, None) == mk.MK_ERR_CUDA, ("write", d, kind, unit)
            assert L.mk_kvq_read(c, P, r, P, 3, unit, None) == mk.MK_ERR_CUDA, ("read", d, kind, unit)
        assert L.mk_kvq_attention(c, P, 4 * d, P, 4 * d, kind, 4, 1, P, 4, P, 1.0, P, 1 << 40, None) == mk.MK_ERR_CUDA
        assert L.mk_kvq_workspace(c, kind, 4, 1, 4000) == 0
"""


def test_calls_without_a_device_return_an_error(lib):
    """Valid arguments where no device answers (a child process that sees none): MK_ERR_CUDA from every call."""
    env = {**os.environ, "CUDA_VISIBLE_DEVICES": "", "PYTHONPATH": ROOT}
    r = subprocess.run([sys.executable, "-c", NO_DEVICE], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])


OVERLAP = """
from persistent_moe_decode_gb300 import mk
L, P, d, hkv = mk.lib(), 1 << 20, 64, 2
def read(unit, count, page, row, head, v=2 * P, hkv=hkv, kind=mk.MK_TYPE_BF16):
    c = mk.mk_kvq_cache(pool=P, num_pages=64, n_kv_heads=hkv, head_dim=d, status=None)
    r = mk.mk_kv_rows(P, v, kind, count, page, row, head)
    w = L.mk_kvq_write(c, r, P, P, 1, unit, None)
    assert w == mk.MK_ERR_CUDA                       # a source may repeat rows; there is no device here
    return L.mk_kvq_read(c, P, r, P, 1, unit, None)
no, ok = mk.MK_ERR_BAD_ARG, mk.MK_ERR_CUDA
# rows: [n][heads][d], [heads][n][d], a fused row, negative strides, one row or one head of any stride
for row, head in ((128, 64), (64, 5 * 64), (1024, 64), (-128, 64), (128, -64), (1024, 512)):
    assert read(1, 5, 0, row, head) == ok, (row, head)
assert read(1, 1, 0, 0, 64) == ok and read(1, 5, 0, 64, 0, hkv=1) == ok and read(1, 0, 0, 0, 64) == ok
for row, head in ((0, 64), (128, 0), (64, 64), (64, 128), (128, 56), (8, 64), (-64, 64), (64, 4 * 64), (2 ** 62, 2 ** 62 + 8)):
    assert read(1, 5, 0, row, head) == no, (row, head)
# pages: [pages][heads][16][d], [pages][16][heads][d], [16][pages][heads][d]
for page, row, head in ((2048, 64, 1024), (2048, 128, 64), (128, 3 * 128, 64), (-2048, 64, 1024)):
    assert read(16, 3, page, row, head) == ok, (page, row, head)
assert read(16, 1, 0, 64, 1024) == ok
for page, row, head in ((0, 64, 1024), (2048, 0, 1024), (2048, 64, 0), (2040, 64, 1024), (1024, 64, 1024), (2048, 64, 64)):
    assert read(16, 3, page, row, head) == no, (page, row, head)
assert read(1, 5, 0, 128, 64, v=P) == no and read(16, 3, 2048, 64, 1024, v=P) == no
"""


def test_a_read_into_rows_that_share_memory_is_refused(lib):
    """Expanded or interleaved destinations, whose content would depend on which thread writes last."""
    env = {**os.environ, "CUDA_VISIBLE_DEVICES": "", "PYTHONPATH": ROOT}
    r = subprocess.run([sys.executable, "-c", OVERLAP], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])


def test_page_bytes_of_heads_the_calls_refuse(lib):
    """mk_kvq_page_bytes supports the shapes that the calls take, and no others."""
    c = mk.mk_kvq_cache(pool=1 << 20, num_pages=4, n_kv_heads=1, head_dim=64, status=None)
    for hkv in (1023, 1024, 1025, 1 << 20, 2 ** 31 - 1):
        c.n_kv_heads = hkv
        taken = lib.mk_kvq_write(c, mk.mk_kv_rows(type=mk.MK_TYPE_BF16), None, None, 0, 1, None) == mk.MK_OK
        assert taken == (hkv <= 1024)
        assert mk.mk_kvq_page_bytes(hkv, 64) == (hkv * 18 * 64 if taken else 0)
        if not taken:
            with pytest.raises(ValueError):
                kvq.page_bytes(hkv, 64)


# ------------------------------------------------ the pools a Decoder is given

def decoder_error(pool, v_pool=None, **cfg):
    from persistent_moe_decode_gb300.configs import TINY

    class Model:
        dims, fp8, embed = TINY, None, torch.zeros(1)
        w_gate = w_up = w_down = None

    with pytest.raises(ValueError) as e:
        mk.Decoder(Model, pool, v_pool, 1, 4, **cfg)
    return str(e.value)


def test_a_decoder_refuses_4_bit_pools_it_would_misread(lib):
    """Another type of one byte, pages that do not lie side by side, another number of layers, a pool that is not on
    the GPU; 4-bit pools beside a v_pool, whose pages a BF16 step would read past their end, and BF16 pools under
    the 4-bit format."""
    from persistent_moe_decode_gb300.configs import TINY as d
    page = mk.mk_kvq_page_bytes(d.n_kv_heads, d.head_dim)
    pools = torch.zeros(d.n_layers, 8, page, dtype=torch.uint8)
    assert "uint8" in decoder_error(pools.to(torch.int8))
    assert "uint8" in decoder_error(pools[:1].expand(d.n_layers + 1, 8, page))
    assert "uint8" in decoder_error(pools[:, :0])
    assert "contiguous" in decoder_error(pools[:, ::2])
    assert "contiguous" in decoder_error(torch.zeros(d.n_layers, 8, 2 * page, dtype=torch.uint8)[..., :page])
    assert "contiguous" in decoder_error(torch.zeros(d.n_layers, page, 8, dtype=torch.uint8).transpose(1, 2))
    assert "contiguous" in decoder_error(pools[:, :1].expand(-1, 8, -1))
    # layers apart are fine, and so is a pool of one page: what remains is where they are
    assert "GPU" in decoder_error(pools) and "GPU" in decoder_error(pools[:, :5]) and "GPU" in decoder_error(pools[:, :1])
    assert "v_pool" in decoder_error(pools, pools)
    bf16 = torch.zeros(d.n_layers, 8, d.n_kv_heads, 16, d.head_dim, dtype=torch.bfloat16)
    assert "v_pool" in decoder_error(bf16, bf16, kv_format=mk.MK_KV_INT4)
