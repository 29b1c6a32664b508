"""Few live sequences among many idle slots of a padded batch, on the GPU."""
from __future__ import annotations

import pytest
import torch

from tests import _kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from persistent_moe_decode_gb300 import build
    build.build()


@pytest.mark.parametrize("slots", [20, 31, 32, 33, 65, 700, 5000])
@pytest.mark.parametrize("grouped", [False, True])
def test_live_sequences_among_idle_slots(slots, grouped):
    """Live ones at the front, at the end, in the middle, next to each other and 31 to 33 slots apart."""
    from persistent_moe_decode_gb300 import kv
    places = {0, 1, slots // 2, slots // 2 + 1, slots - 1} | {x for x in (5 + 31, 5 + 31 + 33, 5 + 31 + 33 + 32) if x < slots}
    for live in (sorted(places), [0], [slots - 1], [slots // 2]):
        news = [0] * slots
        lens = [0] * slots
        for i, b in enumerate(live):
            news[b], lens[b] = (1, 40, 3)[i % 3], (1500, 40, 333)[i % 3]
        st = _kv.batch(news, lens, 2, 64, seed=slots, hq=8)
        want, size = _kv.attention(st["q"], st["k"], st["v"], news, lens, st["tables"])
        cache = kv.PagedCache.from_pools(st["k"], st["v"])
        args = (st["q"], st["starts"], st["tables"], st["lens"])
        if grouped:                                   # a group each
            groups = torch.arange(slots + 1, dtype=torch.int32, device="cuda")
            got = cache.shared_attention(*args, groups, torch.zeros(slots, dtype=torch.int32, device="cuda"))
        else:
            got = cache.attention(*args)
        cache.check()
        assert _kv.attention_off(got, want, size) <= 1
