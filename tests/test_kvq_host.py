"""The 4-bit cache's calls on the host alone (no GPU): where the device cannot
be asked, and what the shape queries answer."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

from persistent_moe_decode_gb300 import build as B
from persistent_moe_decode_gb300 import mk

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
