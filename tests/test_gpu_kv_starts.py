"""Attention over the BF16 paged cache with starts out of order or out of range:
sequences whose rows are theirs alone hold, and all other rows are left as they
were, or NaN, whatever the workspace held before."""
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


def call(starts, lens, groups, prefixes, total):
    """Outputs (7 where nothing was written) of one call with these starts, after a sound one of the same sizes whose
    workspace it takes over, and what the rows of a sequence are due."""
    from persistent_moe_decode_gb300 import kv, mk
    g = torch.Generator(device="cuda")
    g.manual_seed(total)
    batch, hq, hkv, d = len(lens), 4, 2, 64
    pages = batch * 64
    cache = kv.PagedCache(pages, hkv, d)
    cache.k_pool.normal_(generator=g)
    cache.v_pool.normal_(generator=g)
    tables = torch.arange(pages, device="cuda").int().view(batch, 64)
    q = torch.randn(total, hq, d, generator=g, device="cuda").bfloat16()

    def run(starts, groups, prefixes):
        out = torch.full_like(q, 7.0)
        args = (q, vector(starts), tables, vector(lens))
        if groups is None:
            cache.attention(*args, out=out)
        else:
            cache.shared_attention(*args, vector(groups), vector(prefixes), out=out)
        return out
    even = [total * b // batch for b in range(batch + 1)]
    fill = run(even, None if groups is None else [0, batch], [0])
    cache.check()
    assert torch.isfinite(fill).all()
    got = [run(starts, groups, prefixes) for _ in range(3)]
    with pytest.raises(mk.MkError) as e:
        cache.check()
    assert e.value.code == mk.MK_ERR_BAD_ARG
    for x in got[1:]:
        assert torch.equal(x.isnan(), got[0].isnan()) and torch.equal(x.nan_to_num(9.0), got[0].nan_to_num(9.0))

    def want(b):
        lo, hi = starts[b], starts[b + 1]
        table = tables[b:b + 1].clone()
        for i, p in enumerate(prefixes or []):
            if 0 <= groups[i] <= b < groups[i + 1]:
                table[0, :p // 16] = tables[groups[i], :p // 16]
        return slice(lo, hi), _kv.attention(q[lo:hi], cache.k_pool, cache.v_pool, [hi - lo], [lens[b]], table)
    return got[0], want


CASES = [
    # starts, groups, their prefixes, sequences that hold
    ([0, 10, 1000], None, None, [0]),
    ([0, 10, 5, 20], None, None, []),                 # two sequences name rows 5 to 9
    ([3, 9, -4, 12, 20], None, None, [0, 3]),
    ([0, 4, 30, 3, 9, 20], None, None, [4]),          # the second sequence's end lies past the third's start
    ([0, 10, 1000], [0, 1, 2], [64, 64], [0]),        # groups of one sequence each
    ([0, 10, 5, 20], [0, 2, 3], [64, 0], []),
    ([0, 1000, 3, 8, 20], [0, 2, 4], [64, 32], [2, 3]),
    ([0, 1000, 3, 8, 20], [0, 4], [64], [2, 3]),      # one group on both sides of what does not hold
    ([-1, 4, 8, 2000, 20], [0, 1, 3, 4], [0, 0, 0], []),
    ([0, 4, 8, 20], [0, 3, 1, 3], [64, 16, 32], []),  # two groups name sequences 1 and 2
    ([0, 4, 8, 12, 20], [0, 1, -7, 3, 4], [64, 0, 0, 48], [0, 3]),
    ([0, 4, 8, 12, 20], [4, 0, 2, 4], [64, 32, 16], [0, 1, 2, 3]),   # all groups but the first
]


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("starts,groups,prefixes,hold", CASES)
def test_starts_out_of_order(starts, groups, prefixes, hold, many):
    """``many``: behind 400 idle sequences, more tasks than a block has threads."""
    if many:
        n = 400
        starts, hold = [max(starts[0], 0)] * n + list(starts), [b + n for b in hold]
        if groups is not None:
            idle = [0] if groups[0] == 0 else []         # a group of their own, where the others' begin in order
            groups, prefixes = idle + [g + n if g >= 0 else g for g in groups], idle + prefixes
    total = 20
    lens = [200 + 9 * (b % 50) for b in range(len(starts) - 1)]
    got, want = call(starts, lens, groups, prefixes, total)
    held = torch.zeros(total, dtype=torch.bool, device="cuda")
    for b in hold:
        rows, (x, size) = want(b)
        assert _kv.attention_off(got[rows], x, size) <= 1, b
        held[rows] = True
    left = got[~held]
    assert (left.isnan() | (left == 7)).all()
