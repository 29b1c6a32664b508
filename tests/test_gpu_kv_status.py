"""The caches' record of bad indexes on streams of the caller's choice."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from persistent_moe_decode_gb300 import build
    build.build()


def test_paged_cache_flags_on_another_stream_than_its_own():
    """A cache made behind other work on the current stream: what a call on a side stream records at once is still there
    when that work is done."""
    from persistent_moe_decode_gb300 import kv, mk
    pools = torch.zeros(2, 3, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    rope = kv.Rope(64, 1e4)
    x = torch.randn(1, 2, 64, device="cuda")
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([48], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    kv.PagedCache.from_pools(pools[0], pools[1]).append(rope, x, x, x, pos, slots, stream=side)     # all is loaded
    torch.cuda.synchronize()
    torch.cuda._sleep(1_000_000_000)
    cache = kv.PagedCache.from_pools(pools[0], pools[1])
    cache.append(rope, x, x, x, pos, slots, stream=side)
    with pytest.raises(mk.MkError) as e:
        cache.check()
    assert e.value.code == mk.MK_ERR_BAD_PAGE
