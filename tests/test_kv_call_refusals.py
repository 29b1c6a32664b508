"""More of what the paged cache's attention refuses before it touches a device (no
GPU)."""
from __future__ import annotations

import pytest

from persistent_moe_decode_gb300 import build as B
from persistent_moe_decode_gb300 import mk
from tests.test_kv_refusals import P, attn_args, refused


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mk.lib()


@pytest.mark.parametrize("bad", [
    dict(q_starts=P + 2), dict(tables=P + 1), dict(lens=P + 3),
    dict(groups=1, group_starts=P + 2, prefix_lens=P), dict(groups=1, group_starts=P, prefix_lens=P + 2)])
def test_index_arrays_off_their_alignment(lib, bad):
    """Refused for the address: without a device nothing after it would be (and with one no workspace is given)."""
    refused(mk.mk_kv_attention, mk.MK_ERR_BAD_ARG, *attn_args(**bad))


def test_a_workspace_size_that_could_not_be_asked_is_asked_again(monkeypatch):
    """A size of 0 comes of a device query that failed: the call is refused, the next one asks again."""
    import torch
    from persistent_moe_decode_gb300 import kv
    asked, called = [], []

    def size(*args):
        asked.append(args)
        return 0 if len(asked) == 1 else 64

    def attention(c, *args):
        called.append(args)
        if not args[-2]:                                    # workspace_bytes
            raise mk.MkError(mk.MK_ERR_BAD_ARG, "mk_kv_attention")
    monkeypatch.setattr(mk, "mk_kv_workspace", size)
    monkeypatch.setattr(mk, "mk_kv_attention", attention)
    c = kv.PagedCache.__new__(kv.PagedCache)                # on the host: nothing of it is called
    c.k_pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    c.n_kv_heads, c.head_dim, c._dev, c._ws_bytes, c._c = 2, 64, c.k_pool.get_device(), {}, None
    c.status = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    starts, tables, lens = (torch.zeros(n, dtype=torch.int32) for n in (2, 4, 1))

    def call():
        return c._attention(0, q, starts, tables[None], lens, None, None, None, None)
    with pytest.raises(mk.MkError):
        call()
    assert call().shape == q.shape and call().shape == q.shape
    assert len(asked) == 2 and [a[-2] for a in called] == [0, 64, 64]


def test_arrays_that_are_not_read_may_be_anything(lib):
    """Without groups or pages their arrays are not looked at: the refusal is for want of a device, or of a workspace."""
    import torch
    code = mk.MK_ERR_BAD_ARG if torch.cuda.is_available() else mk.MK_ERR_CUDA
    refused(mk.mk_kv_attention, code, *attn_args(group_starts=P + 2, prefix_lens=P + 1))
    refused(mk.mk_kv_attention, code, *attn_args(max_pages=0, tables=P + 2))
