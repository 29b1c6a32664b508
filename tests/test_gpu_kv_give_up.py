"""The paged cache's attention where a wait runs out: the kernels built with limits of
microseconds, which their ordinary waits for copies and products pass.  A block that
gives up ends by itself, flags MK_ERR_TIMEOUT and leaves the GPU as usable as before."""
from __future__ import annotations

import ctypes as C
import os
import subprocess

import pytest
import torch

from tests import _kv

pytestmark = pytest.mark.gpu
LIMITS_NS = (1_000, 3_000, 10_000, 50_000)


@pytest.fixture(scope="module")
def libraries(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from persistent_moe_decode_gb300 import build, mk
    build.build()
    cuda = build._cuda_home()
    tmp = tmp_path_factory.mktemp("kv_give_up")
    jobs = []
    for ns in LIMITS_NS:
        so = tmp / f"kv_{ns}.so"
        jobs.append((ns, so, subprocess.Popen(
            [os.path.join(cuda, "bin", "nvcc"), *build.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-cudart",
             "shared", f"-DMK_KV_WAIT_NS={ns}ull", f"-I{build.INCLUDE}", f"-I{build.CSRC}", "-o", str(so),
             *(os.path.join(build.CSRC, f) for f in ("mk_kv.cu", "mk_kv_attn.cu"))])))
    libs = {}
    for ns, so, job in jobs:
        assert job.wait() == 0
        lib = libs[ns] = C.CDLL(str(so))
        for name in ("mk_kv_workspace", "mk_kv_attention"):
            f = getattr(lib, name)
            f.argtypes, f.restype = getattr(mk.lib(), name).argtypes, getattr(mk.lib(), name).restype
    return libs


@pytest.mark.parametrize("ns", LIMITS_NS)
@pytest.mark.parametrize("hq,hkv,d,news,lens,groups,prefixes", [
    (8, 2, 128, [1, 1, 300], [9000, 200, 2300], None, None),        # narrow and wide items, cut and merged
    (4, 2, 64, [700, 0, 5], [700, 30, 6000], None, None),
    (8, 2, 128, [40, 1, 1], [4200, 4100, 900], [0, 2, 3], [4096, 0])])
def test_a_wait_that_runs_out(libraries, ns, hq, hkv, d, news, lens, groups, prefixes):
    from persistent_moe_decode_gb300 import kv, mk
    st = _kv.batch(news, lens, hkv, d, seed=ns, hq=hq, junk=False)
    if groups:
        st["tables"][1, :256] = st["tables"][0, :256]
    cache = kv.PagedCache.from_pools(st["k"], st["v"])
    q, lib = st["q"], libraries[ns]
    out = torch.empty_like(q)
    n = len(groups) - 1 if groups else 0
    gs, pl = (torch.tensor(x or [0], dtype=torch.int32, device="cuda") for x in (groups, prefixes))
    size = lib.mk_kv_workspace(cache._c, hq, len(q), len(news), n)
    # what lies behind the workspace stays as it is
    ws = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(3):
        rc = lib.mk_kv_attention(cache._c, q.data_ptr(), q.stride(0), out.data_ptr(), out.stride(0), hq, len(q), len(news),
                                 st["starts"].data_ptr(), st["tables"].data_ptr(), st["tables"].shape[1],
                                 st["lens"].data_ptr(), n, gs.data_ptr() if n else None, pl.data_ptr() if n else None,
                                 d ** -0.5, ws.data_ptr(), size, stream)
        assert rc == mk.MK_OK
        torch.cuda.synchronize()
    assert (ws[size:] == 77).all()
    code = int(cache.status.item())
    assert code in (0, mk.MK_ERR_TIMEOUT)
    assert code or ns > 1_000                    # a block plans longer before it copies anything
    # the same call as it is meant, right after
    cache.status.zero_()
    args = (q, st["starts"], st["tables"], st["lens"])
    got = cache.shared_attention(*args, gs, pl) if n else cache.attention(*args)
    cache.check()
    want, size = _kv.attention(q, st["k"], st["v"], news, lens, st["tables"])
    assert _kv.attention_off(got, want, size) <= 1
    if not code:
        assert torch.equal(out, got)
