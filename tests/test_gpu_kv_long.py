"""Long contexts over the BF16 paged cache: every key tile is taken, and once.

In each tile of 128 keys one key outweighs all others, alike in every tile of the
row, and its value has a dim of its own: a result is one over the number of such
keys there.  A tile left out leaves a zero, one taken twice a two-fold.  The keys
stand in 64, 128 tiles at a time, as many as there are dims.

Bounds: all weights of such keys round alike to BF16, 2^-8 against the sum that
takes them unrounded; sums and exponentials in fp32 are off by less than 2^-11; the
result is rounded by 2^-8; the other keys, e^-21 each at most, add less than 2^-13 to
a sum of 1 or more (100,003 of them), and their values are zero.
"""
from __future__ import annotations

import pytest
import torch

from tests import _kv

pytestmark = pytest.mark.gpu
BOUND = 2.0 ** -7 + 2.0 ** -10


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from persistent_moe_decode_gb300 import build
    build.build()


def planted(st, spans, window, d, g):
    """One key in each tile of tiles [window d, window d + d) of spans (table, first token, end): tokens of a page table's
    row whose keys are zero; a tile's key says in its value which of the window's it is."""
    count = 0
    for table, lo, hi in spans:
        n = -(-(hi - lo) // 128)
        tiles = torch.arange(min(window * d, n), min(window * d + d, n), device="cuda")
        if not len(tiles):
            continue
        start = lo + 128 * tiles
        last = torch.clamp(start + 128, max=hi) - start
        at = start + (torch.rand(len(tiles), generator=g, device="cuda") * last).long()
        at[::5] = start[::5]                                             # first and last keys of tiles among them
        at[2::5] = (start + last - 1)[2::5]
        page, row = table[at // 16].long(), at % 16
        st["k"][page, :, row] = 1.0
        st["v"][page, :, row] = torch.nn.functional.one_hot(tiles - window * d, d)[:, None].to(st["v"].dtype)
        count += len(tiles)
    return count


LONG = [
    # hq, hkv, d, new, cached
    (8, 1, 128, 1, 262144),                # many parts, one tile of rows
    (4, 4, 64, 1, 100_003),
    (8, 1, 128, 3, 65_537),
    (16, 1, 64, 70, 70_001),               # wide rows
    (4, 1, 128, 300, 20_011),              # several blocks of rows
    (2, 1, 128, 33, 9_001),
]


@pytest.mark.parametrize("hq,hkv,d,new,length", LONG)
def test_every_tile_of_a_long_context_counts_once(hq, hkv, d, new, length):
    from persistent_moe_decode_gb300 import kv
    g = torch.Generator(device="cuda")
    g.manual_seed(length)
    news, lens = [new, 1], [length, 77]                # beside a short one
    for window in range(-(-length // (128 * d))):
        st = _kv.batch(news, lens, hkv, d, seed=window, hq=hq, junk=False)
        st["q"].fill_(2.625)                           # scores 21 and 29.7 of 64 and 128 dims
        st["k"].zero_()
        st["v"].zero_()
        # keys that every row sees; the last row sees those of the new tokens too
        seen = length - new + 1
        count = planted(st, [(st["tables"][0], 0, seen)], window, d, g)
        cache = kv.PagedCache.from_pools(st["k"], st["v"])
        got = cache.attention(st["q"], st["starts"], st["tables"], st["lens"])[:new]
        cache.check()
        want = torch.zeros(d, dtype=torch.float64, device="cuda")
        if not count:
            continue
        want[:count] = 1 / count
        assert ((got.double() - want).abs() <= BOUND * want).all(), window


@pytest.mark.parametrize("hq,hkv,d,prefix,seqs", [
    (8, 2, 128, 32768, [(1, 33000 + 130 * i) for i in range(16)]),
    (4, 1, 64, 65536 + 48, [(30, 70000), (1, 65536 + 49), (200, 66300)]),
])
def test_every_tile_behind_a_long_prefix_counts_once(hq, hkv, d, prefix, seqs):
    from persistent_moe_decode_gb300 import kv
    g = torch.Generator(device="cuda")
    g.manual_seed(prefix)
    news, lens = [n for n, _ in seqs], [t for _, t in seqs]
    starts = torch.tensor([0] + news).cumsum(0).tolist()
    # the common tiles by windows, then each sequence's own
    for window, own in [(w, None) for w in range(-(-prefix // (128 * d)))] + [(0, b) for b in range(len(seqs))]:
        st = _kv.batch(news, lens, hkv, d, seed=window, hq=hq, prefixes=[prefix], groups=[len(seqs)], junk=False)
        st["q"].fill_(2.625)
        st["k"].zero_()
        st["v"].zero_()
        span = (0, 0, prefix) if own is None else (own, prefix, lens[own] - news[own] + 1)
        count = planted(st, [(st["tables"][span[0]], *span[1:])], window, d, g)
        groups = torch.tensor([0, len(seqs)], dtype=torch.int32, device="cuda")
        cache = kv.PagedCache.from_pools(st["k"], st["v"])
        got = cache.shared_attention(st["q"], st["starts"], st["tables"], st["lens"], groups,
                                     torch.tensor([prefix], dtype=torch.int32, device="cuda"))
        cache.check()
        want = torch.zeros(d, dtype=torch.float64, device="cuda")
        want[:count] = 1 / count
        if own is not None:
            got = got[starts[own]:starts[own + 1]]
        assert ((got.double() - want).abs() <= BOUND * want).all(), (window, own)
