"""The BF16 paged cache's operators at the ends of what their calls take."""
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


def vector(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_the_longest_sequence(new, d):
    """2^28 tokens in 2^24 pages, the same eight pages over and over: as their 128 tokens seen once, but for the new
    tokens, whose own place shortens the last round by less than 40 keys in 2^28."""
    from persistent_moe_decode_gb300 import kv
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    k, v = (torch.randn(8, 1, 16, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(new, 8, d, generator=g, device="cuda").bfloat16()
    tables = (torch.arange(1 << 24, device="cuda") % 8).int()[None]
    cache = kv.PagedCache.from_pools(k, v)
    got = cache.attention(q, vector([0, new]), tables, vector([1 << 28]))
    cache.check()
    # all rows see the eight pages in full
    rows = [_kv.attention(q[i:i + 1], k, v, [1], [128], tables[:, :8]) for i in range(new)]
    want, size = (torch.cat(x) for x in zip(*rows))
    assert _kv.attention_off(got, want, size) <= 1


def test_as_many_sequences_as_there_may_be():
    from persistent_moe_decode_gb300 import kv
    batch, hq, hkv, d = 65535, 4, 1, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    news = torch.randint(0, 3, (batch,), generator=g, device="cuda")
    lens = news + torch.randint(0, 40, (batch,), generator=g, device="cuda")
    starts = torch.cat([torch.zeros(1, device="cuda", dtype=torch.long), news.cumsum(0)]).int()
    pages = 5000
    k, v = (torch.randn(pages, hkv, 16, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    tables = torch.randint(0, pages, (batch, 3), generator=g, device="cuda").int()
    q = torch.randn(int(starts[-1]), hq, d, generator=g, device="cuda").bfloat16()
    cache = kv.PagedCache.from_pools(k, v)
    got = cache.attention(q, starts, tables, lens.int())
    cache.check()
    groups = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    alone = cache.shared_attention(q, starts, tables, lens.int(), groups, torch.zeros(batch, dtype=torch.int32, device="cuda"))
    cache.check()
    picked = [0, 1, 2, 31, 32, 383, 384, 32767, 32768, batch - 2, batch - 1,
              *torch.randint(0, batch, (200,), generator=g, device="cuda").tolist()]
    for b in picked:
        lo, hi, n = int(starts[b]), int(starts[b + 1]), int(lens[b])
        if hi > lo:
            want, size = _kv.attention(q[lo:hi], k, v, [hi - lo], [n], tables[b:b + 1])
            for x in (got, alone):
                assert _kv.attention_off(x[lo:hi], want, size) <= 1
    assert torch.isfinite(got).all() and torch.isfinite(alone).all()


def test_as_many_heads_as_there_may_be():
    from persistent_moe_decode_gb300 import kv
    for hkv, grp in ((1024, 128), (1024, 1), (1, 128)):
        hq, d, news, lens = hkv * grp, 64, [2, 1], [37, 150]
        g = torch.Generator(device="cuda")
        g.manual_seed(hq)
        k, v = (torch.randn(20, hkv, 16, d, generator=g, device="cuda").bfloat16() for _ in range(2))
        tables = torch.randperm(20, generator=g, device="cuda").int().view(2, 10)
        q = torch.randn(3, hq, d, generator=g, device="cuda").bfloat16()
        cache = kv.PagedCache.from_pools(k, v)
        got = cache.attention(q, vector([0, 2, 3]), tables, vector(lens))
        shared = cache.shared_attention(q, vector([0, 2, 3]), tables, vector(lens), vector([0, 1, 2]), vector([16, 96]))
        cache.check()
        for h in {0, 1, hkv // 2, hkv - 1} & set(range(hkv)):
            rows = slice(h * grp, (h + 1) * grp)
            want, size = _kv.attention(q[:, rows], k[:, h:h + 1], v[:, h:h + 1], news, lens, tables)
            for x in (got, shared):
                assert _kv.attention_off(x[:, rows], want, size) <= 1
        assert torch.isfinite(got).all() and torch.isfinite(shared).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_at_any_int32_position(interleaved):
    from persistent_moe_decode_gb300 import kv
    pos = vector([-2 ** 31, -2 ** 31 + 1, -1 << 20, -65537, -1, 0, 1, 2 ** 31 - 1])
    q = torch.randn(8, 3, 128, device="cuda")
    got, _ = kv.Rope(128, 5e5, interleaved=interleaved).apply(q, q[:, :1], pos)
    want, size = _kv.turned(q, pos, 128, 5e5, interleaved)
    assert _kv.rope_off(got, want, size) <= 1
