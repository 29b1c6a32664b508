"""The 4-bit cache's record of bad indexes on streams of the caller's choice."""
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


def test_quant_cache_flags_on_another_stream_than_its_own():
    """A cache made behind other work on the current stream: what a call on a side stream records at once is still there
    when that work is done."""
    from persistent_moe_decode_gb300 import kvq, mk
    pool = kvq.QuantCache(3, 2, 64).pool
    x = torch.randn(1, 2, 64, device="cuda")
    slots = torch.tensor([48], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    kvq.QuantCache.from_pool(pool, 2, 64).write(x, x, slots, stream=side)          # all is loaded
    torch.cuda.synchronize()
    torch.cuda._sleep(1_000_000_000)
    cache = kvq.QuantCache.from_pool(pool, 2, 64)
    cache.write(x, x, slots, stream=side)
    with pytest.raises(mk.MkError) as e:
        cache.check()
    assert e.value.code == mk.MK_ERR_BAD_PAGE
