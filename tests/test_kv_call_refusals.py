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
