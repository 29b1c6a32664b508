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


def test_status_words_are_each_caches_own():
    """Caches made one after the other, more than share a block of words, and one made in a captured graph."""
    from persistent_moe_decode_gb300 import kv, kvq, mk
    pools = torch.zeros(2, 1, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    rope = kv.Rope(64, 1e4)
    x = torch.randn(1, 1, 64, device="cuda")
    pos, past = (torch.tensor([v], dtype=torch.int32, device="cuda") for v in (0, 16))
    caches = [kv.PagedCache.from_pools(pools[0], pools[1]) for _ in range(1500)]
    quant = kvq.QuantCache(1, 1, 64)
    assert len({c.status.data_ptr() for c in caches} | {quant.status.data_ptr()}) == 1501
    caches[3].append(rope, x, x, x, pos, past)
    quant.write(x, x, past)
    for c in (caches[3], quant):
        with pytest.raises(mk.MkError):
            c.check()
    for c in caches:
        assert c.status.shape == (1,)
    assert sum(int(c.status) for c in caches[::100]) == 0 and int(caches[3].status) == 0
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            inside = kv.PagedCache.from_pools(pools[0], pools[1])
            inside.append(rope, x, x, x, pos, past)
    graph.replay()
    with pytest.raises(mk.MkError):
        inside.check()
    caches[4].check()


def test_status_words_made_in_inference_mode_are_cleared_outside():
    from persistent_moe_decode_gb300 import kv, mk
    pools = torch.zeros(2, 1, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    rope = kv.Rope(64, 1e4)
    x = torch.randn(1, 1, 64, device="cuda")
    pos, past = (torch.tensor([v], dtype=torch.int32, device="cuda") for v in (0, 16))
    mk._words.clear()                                     # the next block of words is made in there
    with torch.inference_mode():
        first = kv.PagedCache.from_pools(pools[0], pools[1])
    second = kv.PagedCache.from_pools(pools[0], pools[1])
    for c in (first, second):
        for _ in range(2):
            c.append(rope, x, x, x, pos, past)
            with pytest.raises(mk.MkError):
                c.check()
        c.check()
