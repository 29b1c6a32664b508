"""The 4-bit cache's calls as a program makes them beside others: other streams,
shared or overlapping buffers, the ends of the ranges that include/mk.h gives."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from persistent_moe_decode_gb300 import mk
from persistent_moe_decode_gb300.kvq import QuantCache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from persistent_moe_decode_gb300 import build
    build.build()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_the_workspace_of_arguments_that_the_attention_refuses_is_none():
    """mk_kvq_workspace is 0 where mk_kvq_attention refuses the same type, heads, batch or page tables."""
    c = QuantCache(4, 2, 64)
    q = torch.zeros(1, 4, 64, device="cuda")
    ln = ints(1)
    fits = dict(kind=mk.MK_TYPE_F32, hq=4, batch=1, pages=1 << 20)
    assert mk.mk_kvq_workspace(c._c, *fits.values()) > 0
    for bad in (dict(kind=2), dict(kind=-1), dict(pages=-1), dict(pages=1 << 27), dict(pages=2 ** 31 - 1), dict(hq=3),
                dict(batch=65536)):
        kw = {**fits, **bad}
        assert mk.mk_kvq_workspace(c._c, *kw.values()) == 0, bad
        with pytest.raises(mk.MkError):              # refused before anything is read
            mk.mk_kvq_attention(c._c, q.data_ptr(), 256, q.data_ptr(), 256, kw["kind"], kw["hq"], kw["batch"],
                                ln.data_ptr(), kw["pages"], ln.data_ptr(), 1.0, q.data_ptr(), 1 << 40)


@pytest.mark.parametrize("given", [True, False], ids=["stream argument", "current stream"])
def test_check_sees_calls_that_have_not_run_yet_on_another_stream(given):
    """A call behind long work on a stream of its own: check() on the current stream waits for it, and the record it
    clears stays cleared."""
    hkv, d = 2, 64
    c = QuantCache(4, hkv, d)
    k = torch.zeros(1, hkv, d, dtype=torch.bfloat16, device="cuda")
    bad, good = ints(64), ints(5)
    side = torch.cuda.Stream()
    c.write(k, k, good)                              # loading a kernel may wait for the device
    for slots in (bad, good, bad):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)           # a tenth of a second
            if not given:
                c.write(k, k, slots)
        if given:
            c.write(k, k, slots, stream=side)
        assert not side.query()
        if slots is good:
            c.check()
        else:
            with pytest.raises(mk.MkError) as e:
                c.check()
            assert e.value.code == mk.MK_ERR_BAD_PAGE
        assert side.query()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hkv,grp,d,wide", [(4, 1, 64, 8), (1, 8, 128, 8), (2, 9, 64, 3000), (4, 8, 128, 3000)],
                         ids=["cluster64", "cluster128", "two kernels, tiles", "two kernels"])
def test_the_output_over_the_query_where_rows_of_several_tasks_share_a_cache_line(hkv, grp, d, wide, dtype):
    """out is q, at an offset of 16 bytes and with rows that are no multiple of 128 bytes apart: the bits are those of
    a separate output, and what lies between and behind the rows stays."""
    gen = torch.Generator("cuda").manual_seed(d + hkv)
    batch, hq, pages = 9, hkv * grp, 40
    c = QuantCache(pages, hkv, d)
    k, v = (torch.randn(pages, hkv, 16, d, device="cuda", generator=gen).bfloat16() for _ in range(2))
    ids = torch.arange(pages, dtype=torch.int32, device="cuda")
    c.write_pages(k, v, ids, ids)
    table = torch.randint(0, pages, (batch, wide), device="cuda", generator=gen).int()
    lens = ints(1, 0, 128, 77, 16, 5, 100, 33, 64)
    unit = 16 // dtype.itemsize
    stride = hq * d + unit
    flat = torch.randn(unit + batch * stride, device="cuda", generator=gen).to(dtype)
    q = flat[unit:].view(batch, stride)[:, :hq * d].unflatten(1, (hq, d))
    want = c.attention(q, table, lens)
    for _ in range(5):
        both = flat.clone()
        same = both[unit:].view(batch, stride)[:, :hq * d].unflatten(1, (hq, d))
        assert c.attention(same, table, lens, out=same).data_ptr() == same.data_ptr()
        assert torch.equal(same, want)
        same.copy_(q)
        assert torch.equal(both, flat)
    c.check()


def test_a_stream_of_another_device_is_refused():
    """It would make its device current, and the kernels would run there on this device's addresses."""
    class Stream:                                    # stands in for a stream of a second GPU
        device = torch.device("cuda", torch.cuda.current_device() + 1)

    hkv, d = 2, 64
    c = QuantCache(4, hkv, d)
    k = torch.zeros(1, hkv, d, dtype=torch.bfloat16, device="cuda")
    pools = torch.zeros(4, hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    other = pools.clone()
    one = ints(1)
    for call in (lambda st: c.write(k, k, one, stream=st), lambda st: c.read(one, stream=st),
                 lambda st: c.write_pages(pools, pools, one, one, stream=st),
                 lambda st: c.read_pages(one, pools, other, one, stream=st),
                 lambda st: c.attention(k, one[None], one, stream=st)):
        with pytest.raises(ValueError, match="stream"):
            call(Stream)
        call(torch.cuda.Stream())
        torch.cuda.synchronize()
    c.check()


def test_read_pages_into_pools_that_share_memory_is_refused():
    hkv, d = 2, 64
    c = QuantCache(4, hkv, d)
    k, v = (torch.full((4, hkv, 16, d), x, device="cuda") for x in (2.0, 3.0))
    ids = ints(0, 1)
    for a, b in ((k, k), (k[:1].expand(4, -1, -1, -1), v[:1].expand(4, -1, -1, -1)),
                 (k[:, :1].expand(-1, hkv, -1, -1), v[:, :1].expand(-1, hkv, -1, -1))):
        with pytest.raises(mk.MkError) as e:
            c.read_pages(ids, a, b, ids)
        assert e.value.code == mk.MK_ERR_BAD_ARG
    assert (k == 2).all() and (v == 3).all()
    both = torch.full((4, hkv, 2, 16, d), 5.0, device="cuda")    # keys and values side by side lie apart
    c.read_pages(ids, both[:, :, 0], both[:, :, 1], ids)
    assert (both[:2] == 0).all() and (both[2:] == 5).all()
    c.write_pages(k[:1].expand(4, -1, -1, -1), k[:1].expand(4, -1, -1, -1), ints(0, 1, 2, 3), ints(0, 1, 2, 3))
    c.read_pages(ints(0, 1, 2, 3), k, v, ints(0, 1, 2, 3))
    assert (k == 2).all() and (v == 2).all()
    c.check()
