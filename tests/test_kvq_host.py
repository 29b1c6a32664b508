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
        r = mk.mk_kv_rows(P, P, kind, 64, 64 * d, d, 16 * d)
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
