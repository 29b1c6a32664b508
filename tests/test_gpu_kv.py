"""The BF16 paged cache's operators on the GPU against their definitions in 64
bits: rotary positions, rows into the cache, attention over packed prompts and
over shared prefixes."""
from __future__ import annotations

import math

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


def kv():
    from persistent_moe_decode_gb300 import kv
    return kv


# ------------------------------------------------------------------ rotary

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,r", [
    (1, 1, 1, 64, 64), (1, 32, 4, 128, 128), (5, 3, 1, 64, 16), (13, 4, 2, 128, 32), (150, 10, 5, 128, 112),
    (1217, 8, 8, 64, 48), (4100, 16, 4, 128, 128)])
def test_rope(n, hq, hkv, d, r, interleaved, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(n + r)
    x = torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda").to(dtype)
    q, k, _ = x.split([hq, hkv, hkv], 1)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda").int()
    pos[0], pos[-1] = 0, 2 ** 31 - 1 if n > 2 else 262143
    before = x.clone()
    rope = kv().Rope(d, 1e6, rotary_dim=r, interleaved=interleaved)
    got = rope.apply(q, k, pos)
    assert torch.equal(x, before)
    for y, t in zip(got, (q, k)):
        assert y.dtype is dtype and y.is_contiguous()
        want, size = _kv.turned(t, pos, r, 1e6, interleaved)
        assert _kv.rope_off(y, want, size) <= 1
        assert torch.equal(y[..., r:], t[..., r:])
    # in place, on the strided rows of the projection
    rope.apply(q, k, pos, out=(q, k))
    assert torch.equal(q, got[0]) and torch.equal(k, got[1]) and torch.equal(x[:, hq + hkv:], before[:, hq + hkv:])


@pytest.mark.parametrize("scaling,factor", [("linear", 4.0), ("ntk", 8.0), ("yarn", 32.0)])
def test_rope_scaled(scaling, factor):
    d, r, theta, ctx = 128, 64, 1e4, 4096
    pos = torch.tensor([0, 1, 4095, 4096, 131071, 1 << 20], device="cuda").int()
    q = torch.randn(6, 4, d, device="cuda")
    rope = kv().Rope(d, theta, rotary_dim=r, scaling=scaling, factor=factor, original_context=ctx)
    f, m = [], 1.0
    for i in range(r // 2):
        x = theta ** (-2 * i / r)
        if scaling == "linear":
            x /= factor
        if scaling == "ntk":
            x = (theta * factor ** (r / (r - 2))) ** (-2 * i / r)
        if scaling == "yarn":
            lo = max(0, math.floor(r * math.log(ctx / (32 * 2 * math.pi)) / (2 * math.log(theta))))
            hi = min(r - 1, math.ceil(r * math.log(ctx / (2 * math.pi)) / (2 * math.log(theta))))
            w = min(1, max(0, (i - lo) / max(hi - lo, 1e-3)))
            x, m = x * (w / factor + 1 - w), 1 + 0.1 * math.log(factor)
        f.append(x)
    want, size = _kv.turned(q, pos, r, theta, False, f, m)
    got, _ = rope.apply(q, q[:, :1], pos)
    assert _kv.rope_off(got, want, size) <= 1


def test_rope_nothing():
    rope = kv().Rope(64, 1e4)
    pos = torch.zeros(0, dtype=torch.int32, device="cuda")
    q, k = rope.apply(torch.zeros(0, 4, 64, device="cuda"), torch.zeros(0, 2, 64, device="cuda"), pos)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    pos = torch.tensor([7], device="cuda").int()
    q, k = rope.apply(torch.zeros(1, 0, 64, device="cuda"), torch.ones(1, 2, 64, device="cuda"), pos)
    want, size = _kv.turned(torch.ones(1, 2, 64, device="cuda"), pos, 64, 1e4, False)
    assert _kv.rope_off(k, want, size) <= 1


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,hq,hkv,d,r,interleaved", [
    (1, 4, 2, 64, 64, False), (17, 32, 4, 128, 128, False), (333, 6, 3, 64, 32, True), (2999, 16, 4, 128, 128, False)])
def test_append(n, hq, hkv, d, r, interleaved, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    pages = -(-n // 16) + 2
    cache = kv().PagedCache(pages, hkv, d)
    cache.k_pool.normal_(generator=g)
    cache.v_pool.normal_(generator=g)
    k0, v0 = cache.k_pool.clone(), cache.v_pool.clone()
    x = torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda").to(dtype)
    q, k, v = x.split([hq, hkv, hkv], 1)
    pos = torch.randint(0, 1 << 18, (n,), generator=g, device="cuda").int()
    slots = torch.randperm(pages * 16, generator=g, device="cuda")[:n].int()
    if n > 4:
        slots[2], slots[-2] = -1, -(1 << 31)
    rope = kv().Rope(d, 1e5, rotary_dim=r, interleaved=interleaved)
    out = cache.append(rope, q, k, v, pos, slots)
    cache.check()
    assert out.dtype is torch.bfloat16
    want, size = _kv.turned(q, pos, r, 1e5, interleaved)
    assert _kv.rope_off(out, want, size) <= 1
    want, size = _kv.turned(k, pos, r, 1e5, interleaved)
    live = (slots >= 0).nonzero().flatten()
    s = slots[live].long()
    assert _kv.rope_off(cache.k_pool[s // 16, :, s % 16], want[live], size[live]) <= 1
    assert torch.equal(cache.v_pool[s // 16, :, s % 16], v[live].bfloat16())
    k0[s // 16, :, s % 16] = cache.k_pool[s // 16, :, s % 16]
    v0[s // 16, :, s % 16] = cache.v_pool[s // 16, :, s % 16]
    assert torch.equal(k0, cache.k_pool) and torch.equal(v0, cache.v_pool)


def test_append_past_the_cache_is_flagged_and_skipped():
    from persistent_moe_decode_gb300 import mk
    cache = kv().PagedCache(3, 2, 64)
    rope = kv().Rope(64, 1e4)
    x = torch.randn(3, 2, 64, device="cuda")
    pos = torch.arange(3, device="cuda").int()
    cache.append(rope, x, x, x, pos, torch.tensor([48, 2 ** 31 - 1, 47], device="cuda").int())
    with pytest.raises(mk.MkError) as e:
        cache.check()
    assert e.value.code == mk.MK_ERR_BAD_PAGE
    cache.check()
    assert torch.equal(cache.v_pool[2, :, 15], x[2].bfloat16())
    assert int((cache.v_pool != 0).any(-1).sum()) == 2


# --------------------------------------------------------------- attention

def run(st, scale=None, out=None):
    cache = kv().PagedCache.from_pools(st["k"], st["v"])
    got = cache.attention(st["q"], st["starts"], st["tables"], st["lens"], scale=scale, out=out)
    cache.check()
    return got


PROMPTS = [
    # hq, hkv, d, new tokens, cached tokens (the new ones included)
    (1, 1, 64, [1], [1]),
    (4, 2, 64, [64], [64]),
    (8, 1, 128, [1], [129]),
    (8, 8, 128, [127, 1, 128], [127, 128, 128]),
    (32, 4, 128, [1, 1, 1, 1], [1, 16, 17, 3000]),
    (32, 4, 128, [31, 0, 33, 32], [31, 40, 33, 1000]),
    (5, 1, 64, [200, 51], [200, 1511]),
    (9, 3, 128, [300], [555]),
    (14, 2, 128, [77, 1, 19], [1200, 900, 19]),
    (16, 4, 128, [1000, 257], [1000, 2305]),
    (128, 1, 64, [3, 9], [3, 260]),
    (64, 1, 128, [130], [700]),
    (16, 16, 64, [513], [513]),
    (32, 4, 128, [2048], [2048]),
    (4, 2, 64, [5000], [5000]),
    (2, 1, 128, [1, 40], [9000, 20011]),
]


@pytest.mark.parametrize("hq,hkv,d,news,lens", PROMPTS)
def test_attention(hq, hkv, d, news, lens):
    st = _kv.batch(news, lens, hkv, d, seed=sum(lens), hq=hq)
    got = run(st)
    want, size = _kv.attention(st["q"], st["k"], st["v"], news, lens, st["tables"])
    assert _kv.attention_off(got, want, size) <= 1
    assert torch.equal(run(st), got)


@pytest.mark.parametrize("seed", range(6))
def test_attention_ragged_batches(seed):
    import random
    rng = random.Random(seed)
    hkv, grp, d = rng.choice([1, 2, 3]), rng.choice([1, 2, 3, 6, 7, 8]), rng.choice([64, 128])
    news = [rng.choice([0, 1, rng.randrange(1, 300)]) for _ in range(rng.randrange(1, 40))]
    lens = [n + rng.choice([0, rng.randrange(0, 2000)]) for n in news]
    st = _kv.batch(news, lens, hkv, d, seed=seed, hq=hkv * grp)
    want, size = _kv.attention(st["q"], st["k"], st["v"], news, lens, st["tables"], scale=0.3)
    assert _kv.attention_off(run(st, scale=0.3), want, size) <= 1


def test_attention_rows_that_see_nothing():
    """More new tokens than cached ones: the first rows come before the first key."""
    for news, lens in (([5], [3]), ([300], [10]), ([40, 2], [0, 2]), ([513], [200])):
        st = _kv.batch(news, lens, 2, 64, seed=1, hq=8)
        got = run(st)
        want, size = _kv.attention(st["q"], st["k"], st["v"], news, lens, st["tables"])
        assert _kv.attention_off(got, want, size) <= 1
        assert (got[:news[0] - lens[0]] == 0).all()


def test_attention_rows_of_no_sequence_stay():
    st = _kv.batch([7, 70], [100, 70], 2, 128, seed=3, hq=8)
    for lo, hi in ((0, 5), (4, 0)):
        q = torch.cat([torch.full((lo, 8, 128), math.nan, device="cuda").bfloat16(), st["q"],
                       torch.full((hi, 8, 128), math.nan, device="cuda").bfloat16()])
        out = torch.full_like(q, 7.0)
        st2 = dict(st, q=q, starts=st["starts"] + lo)
        run(st2, out=out)
        want, size = _kv.attention(st["q"], st["k"], st["v"], [7, 70], [100, 70], st["tables"])
        assert _kv.attention_off(out[lo:lo + 77], want, size) <= 1
        assert (out[:lo] == 7).all() and (out[lo + 77:] == 7).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,length", [(200, 200), (150, 700), (1, 300)])
def test_attention_hidden_infinities(new, length, d):
    """NaN and infinities among keys and values reach the rows that see them, and no others."""
    st = _kv.batch([new], [length], 2, d, seed=5, hq=4)
    at = lambda t: (int(st["tables"][0, t // 16]), t % 16)  # noqa: E731
    first = length - new
    marks = [(length - 1, math.inf, 3), (first + new // 2, math.nan, 5), (first + new // 2 + 1, -math.inf, 5),
             (first + new // 3, -math.inf, d - 1)]
    for t, x, i in marks:
        p, r = at(t)
        st["v"][p, 0, r, i] = x
    p, r = at(length - 1)
    st["k"][p, 1, r, 0] = math.nan
    got = run(st)
    want, size = _kv.attention(st["q"], st["k"], st["v"], [new], [length], st["tables"])
    assert _kv.attention_off(got, want, size) <= 1
    if new > 10:
        assert torch.isfinite(got[:new // 3]).all() and torch.isfinite(got[:new - 1, 2:]).all()


def test_attention_large_and_small_scores():
    """Scores far apart, growing along the sequence (the running maximum moves in every tile) and falling."""
    for sign in (1, -1):
        st = _kv.batch([64], [1500], 1, 64, seed=8, hq=2, junk=False)
        t = torch.arange(1500, device="cuda")
        k = torch.randn(1500, 64, device="cuda") * 0.1 + sign * (t[:, None] / 100.0)
        st["k"][st["tables"][0, t // 16].long(), 0, t % 16] = k.bfloat16()
        st["q"] = (torch.rand_like(st["q"].float()) * 0.5 + 0.2).bfloat16()
        want, size = _kv.attention(st["q"], st["k"], st["v"], [64], [1500], st["tables"])
        assert _kv.attention_off(run(st), want, size) <= 1


def test_attention_bad_sequences_are_nan_and_flagged():
    from persistent_moe_decode_gb300 import mk
    def fresh():
        st = _kv.batch([3, 40, 2], [300, 200, 50], 2, 64, seed=9, hq=4, spare=3)
        want, size = _kv.attention(st["q"], st["k"], st["v"], [3, 40, 2], [300, 200, 50], st["tables"])
        return st, want, size
    for what, code in (("page", mk.MK_ERR_BAD_PAGE), ("negative page", mk.MK_ERR_BAD_PAGE),
                       ("long", mk.MK_ERR_BAD_ARG), ("negative", mk.MK_ERR_BAD_ARG)):
        st, want, size = fresh()
        if what == "page":
            st["tables"][1, 0] = st["k"].shape[0]
        elif what == "negative page":
            st["tables"][1, 0] = -1
        else:
            st["lens"][1] = -1 if what == "negative" else st["tables"].shape[1] * 16 + 1
        cache = kv().PagedCache.from_pools(st["k"], st["v"])
        got = cache.attention(st["q"], st["starts"], st["tables"], st["lens"])
        with pytest.raises(mk.MkError) as e:
            cache.check()
        assert e.value.code == code
        assert got[3:43].isnan().all(), what
        for s in (slice(0, 3), slice(43, 45)):
            assert _kv.attention_off(got[s], want[s], size[s]) <= 1
    # starts that decrease or leave the rows: no access outside, the other sequences hold
    for i, x in ((1, 50), (3, 1000), (0, -5), (2, 1)):
        st, want, size = fresh()
        st["starts"][i] = x
        cache = kv().PagedCache.from_pools(st["k"], st["v"])
        got = cache.attention(st["q"], st["starts"], st["tables"], st["lens"])
        with pytest.raises(mk.MkError) as e:
            cache.check()
        assert e.value.code == mk.MK_ERR_BAD_ARG
        if i in (0, 3):
            s = slice(43, 45) if i == 0 else slice(0, 3)
            assert _kv.attention_off(got[s], want[s], size[s]) <= 1


def test_attention_strided_rows_and_in_place():
    news, lens = [33, 90], [500, 90]
    st = _kv.batch(news, lens, 2, 128, seed=11, hq=8)
    want, size = _kv.attention(st["q"], st["k"], st["v"], news, lens, st["tables"])
    wide = torch.randn(123, 12, 128, device="cuda").bfloat16()
    wide[:, :8] = st["q"]
    keep = wide[:, 8:].clone()
    got = run(dict(st, q=wide[:, :8]))
    assert _kv.attention_off(got, want, size) <= 1
    # rows of another order of dims, an odd address: copied first
    assert torch.equal(run(dict(st, q=st["q"].transpose(0, 1).contiguous().transpose(0, 1))), got)
    odd = torch.empty(123 * 8 * 128 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(123, 8, 128).copy_(st["q"])
    assert torch.equal(run(dict(st, q=odd)), got)
    # tables and lengths as views
    wide_t = torch.full((2, 2 * st["tables"].shape[1]), -9, dtype=torch.int32, device="cuda")
    wide_t[:, ::2] = st["tables"]
    assert torch.equal(run(dict(st, tables=wide_t[:, ::2])), got)
    out = run(dict(st, q=wide[:, :8]), out=wide[:, :8])
    assert torch.equal(out, got) and torch.equal(wide[:, :8], got) and torch.equal(wide[:, 8:], keep)


def test_attention_many_sequences():
    """More tasks than a warp has lanes, than a block has threads, and several to a thread."""
    import random
    rng = random.Random(2)
    for batch in (33, 390, 1500):
        news = [rng.choice([0, 1, 1, 1, 2, 37]) for _ in range(batch)]
        lens = [n + rng.choice([0, 3, 130, 500]) for n in news]
        lens[batch // 2] = 6000
        st = _kv.batch(news, lens, 1, 64, seed=batch, hq=4)
        want, size = _kv.attention(st["q"], st["k"], st["v"], news, lens, st["tables"])
        assert _kv.attention_off(run(st), want, size) <= 1


def test_attention_without_pages():
    st = _kv.batch([3, 1], [0, 0], 2, 64, seed=1, hq=4, spare=0)
    assert st["tables"].shape == (2, 0)
    assert (run(st) == 0).all()
    empty = dict(st, q=st["q"][:0], starts=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert run(empty).shape == (0, 4, 64)


def test_attention_far_pages():
    """Pages whose elements lie past 2^31: the last ones of a cache of 4.5 GB each of keys and values."""
    hkv, d, pages = 8, 128, 140_000
    k = torch.empty(pages, hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    n = 700
    ids = torch.cat([torch.arange(pages - 40, pages), torch.arange(0, 4)]).int().cuda()
    for p in (k, v):
        p[ids.long()] = torch.randn(44, hkv, 16, d, generator=g, device="cuda").bfloat16()
    assert k.numel() > 1 << 31
    st = dict(k=k, v=v, q=torch.randn(100, 16, d, generator=g, device="cuda").bfloat16(), tables=ids[None].contiguous(),
              starts=torch.tensor([0, 100], dtype=torch.int32, device="cuda"),
              lens=torch.tensor([n], dtype=torch.int32, device="cuda"))
    want, size = _kv.attention(st["q"], k, v, [100], [n], st["tables"])
    assert _kv.attention_off(run(st), want, size) <= 1
    # the cache's rows there, written
    cache = kv().PagedCache.from_pools(k, v)
    x = torch.randn(2, 3 * hkv, d, generator=g, device="cuda").bfloat16()
    pos = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    slots = torch.tensor([pages * 16 - 1, 17], dtype=torch.int32, device="cuda")
    cache.append(kv().Rope(d, 1e4), *x.split(hkv, 1), pos, slots)
    cache.check()
    assert torch.equal(v[pages - 1, :, 15], x[0, 2 * hkv:]) and torch.equal(v[1, :, 1], x[1, 2 * hkv:])


def test_far_strides():
    """Rows 2^30 elements apart."""
    wide = torch.empty((2 << 30) + 4096, dtype=torch.bfloat16, device="cuda")
    rows = wide.as_strided((3, 4, 64), (1 << 30, 64, 1))
    st = _kv.batch([3], [150], 2, 64, seed=4, hq=4)
    want, size = _kv.attention(st["q"], st["k"], st["v"], [3], [150], st["tables"])
    rows.copy_(st["q"])
    out = wide.as_strided((3, 4, 64), (1 << 30, 64, 1), 1024)
    run(dict(st, q=rows), out=out)
    assert _kv.attention_off(out.clone(), want, size) <= 1
    pos = torch.tensor([3, 70000, 9], dtype=torch.int32, device="cuda")
    got, _ = kv().Rope(64, 1e4).apply(rows, rows[:, :1], pos)
    want, size = _kv.turned(st["q"], pos, 64, 1e4, False)
    assert _kv.rope_off(got, want, size) <= 1


# ------------------------------------------------------------------ shared

SHARED = [
    # hq, hkv, d, groups: (common tokens, [(new, cached), ...])
    (4, 2, 64, [(64, [(1, 81), (1, 65), (0, 70)]), (0, [(5, 9), (1, 33)])]),
    (32, 4, 128, [(2048, [(1, 2049 + 37 * i) for i in range(16)])]),
    (32, 4, 128, [(16, [(1, 17)])]),
    (8, 1, 128, [(4096, [(20, 4116), (1, 4097), (50, 4200), (0, 4096)]), (0, []), (128, [(1, 129), (3, 200)])]),
    (5, 1, 64, [(1600, [(9, 1609)] * 7), (48, [(2, 50), (2, 300)])]),
    (16, 16, 64, [(512, [(1, 600)] * 40)]),
    (6, 2, 128, [(0, [(100, 100), (1, 900)]), (0, [(7, 7)])]),
    (128, 1, 64, [(304, [(1, 305), (2, 333)])]),
]


def shared_batch(hq, hkv, d, groups, seed, **kw):
    news = [n for _, s in groups for n, _ in s]
    lens = [t for _, s in groups for _, t in s]
    counts, prefixes = [len(s) for _, s in groups], [p for p, _ in groups]
    st = _kv.batch(news, lens, hkv, d, seed, hq, prefixes, counts, **kw)
    starts = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    first = [int(starts[g]) for g, c in enumerate(counts) for _ in range(c)]
    per = [prefixes[g] for g, c in enumerate(counts) for _ in range(c)]
    want, size = _kv.attention(st["q"], st["k"], st["v"], news, lens, st["tables"], None, per, first)
    st.update(group_starts=starts, prefix_lens=torch.tensor(prefixes, dtype=torch.int32, device="cuda"))
    return st, want, size


def run_shared(st, **kw):
    cache = kv().PagedCache.from_pools(st["k"], st["v"])
    got = cache.shared_attention(st["q"], st["starts"], st["tables"], st["lens"], st["group_starts"], st["prefix_lens"],
                                 **kw)
    return got, cache


@pytest.mark.parametrize("hq,hkv,d,groups", SHARED)
def test_shared_attention(hq, hkv, d, groups):
    st, want, size = shared_batch(hq, hkv, d, groups, seed=13)
    got, cache = run_shared(st)
    cache.check()
    assert _kv.attention_off(got, want, size) <= 1
    assert torch.equal(run_shared(st)[0], got)
    q = st["q"].clone()
    out, _ = run_shared(dict(st, q=q), out=q)
    assert torch.equal(out, got)


def test_shared_attention_bad_groups():
    from persistent_moe_decode_gb300 import mk
    groups = [(64, [(1, 81), (2, 66)]), (32, [(5, 50), (1, 33)])]

    def case(change, code, nan_rows, only=None):
        st, want, size = shared_batch(4, 2, 64, groups, seed=17)
        change(st)
        q = st["q"]
        got, cache = run_shared(st, out=torch.zeros_like(q))
        with pytest.raises(mk.MkError) as e:
            cache.check()
        assert e.value.code == code
        assert got[nan_rows].isnan().all()
        rest = only or [i for i in range(9) if i not in range(9)[nan_rows]]
        assert _kv.attention_off(got[rest], want[rest], size[rest]) <= 1

    def put(name, i, x):
        def f(st):
            st[name][i] = x
        return f
    case(put("prefix_lens", 0, 40), mk.MK_ERR_BAD_ARG, slice(0, 3))          # no whole pages
    case(put("prefix_lens", 0, -16), mk.MK_ERR_BAD_ARG, slice(0, 3))
    case(put("prefix_lens", 1, 48), mk.MK_ERR_BAD_ARG, slice(3, 9))          # reaches into the new tokens
    case(put("prefix_lens", 1, 1 << 30), mk.MK_ERR_BAD_ARG, slice(3, 9))
    case(put("group_starts", 2, 3), mk.MK_ERR_BAD_ARG, slice(8, 9))          # the last sequence is in no group
    case(put("tables", (0, 1), 1 << 20), mk.MK_ERR_BAD_PAGE, slice(0, 3))    # a common page
    case(put("tables", (2, 2), -1), mk.MK_ERR_BAD_PAGE, slice(3, 8))         # one sequence's own page
    case(put("group_starts", 2, 7), mk.MK_ERR_BAD_ARG, slice(3, 9))          # past the batch
    case(put("group_starts", 1, -1), mk.MK_ERR_BAD_ARG, slice(0, 9))         # no groups left
    # starts that go up and down again: the rows of the sequence before them hold
    case(put("starts", 2, 9), mk.MK_ERR_BAD_ARG, slice(9, 9), only=[0])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("slope", [0.0, 0.01, -0.01])
def test_parts_on_both_sides_of_the_merge_rule(d, slope):
    """Long keys for just as many rows (of heads) as four parts at a time are added up for, and for one more: parts of
    like and of far apart maxima.  A NaN among values, one among keys, whose weights round to zero beside others, reach
    the rows that see them; scores of -infinity alone have no weight, and a row of nothing else is NaN."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for rows in (2 * sms, 2 * sms + 1):
        groups = [(4096, [(rows - 2, 6000), (1, 4400)]), (0, [(1, 700)])]
        news, lens = [rows - 2, 1, 1], [6000, 4400, 700]
        st, _, _ = shared_batch(32, 4, d, groups, seed=rows, junk=False)

        def keys(b, lo, n):
            t = torch.arange(lo, n, device="cuda")
            return st["tables"][b, t // 16].long(), t % 16, (slope * t)[:, None, None].bfloat16()
        for b, lo in ((0, 0), (1, 4096), (2, 0)):
            page, row, up = keys(b, lo, lens[b])
            st["k"][page, :, row] += up
        st["q"].copy_((torch.rand_like(st["q"].float()) * 0.5 + 0.2).bfloat16())
        page, row, _ = keys(0, 5998, 6000)
        st["v"][page[0], 1, row[0], 7] = math.nan            # of the last two tokens' 8 heads
        page, row, _ = keys(0, 5990, 5991)
        st["k"][page, 2, row, 0] = math.nan                  # of the last ten tokens'
        for b, lo in ((1, 4096), (2, 0)):
            page, row, _ = keys(b, lo, lens[b])
            st["k"][page, 3, row, 0] = -math.inf
        tables = st["tables"].clone()
        tables[1, :256] = tables[0, :256]
        want, size = _kv.attention(st["q"], st["k"], st["v"], news, lens, tables)
        assert want.isnan().sum() == 2 * 8 + 10 * 8 * d + 8 * d
        got, cache = run_shared(st)
        cache.check()
        assert _kv.attention_off(got, want, size) <= 1
        assert _kv.attention_off(run(dict(st, tables=tables)), want, size) <= 1


# ---------------------------------------------------- streams, graphs, devices

def test_calls_on_a_side_stream_and_in_a_graph():
    m = kv()
    news, lens = [1, 40, 1], [700, 340, 4000]
    st = _kv.batch(news, lens, 2, 128, seed=21, hq=16)
    want, size = _kv.attention(st["q"], st["k"], st["v"], news, lens, st["tables"])
    cache = m.PagedCache.from_pools(st["k"], st["v"])
    base = run(st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cache.attention(st["q"], st["starts"], st["tables"], st["lens"], stream=side)
    side.synchronize()
    assert torch.equal(got, base)
    # a rotary call, an append and an attention captured together, replayed with other inputs
    rope = m.Rope(128, 1e4)
    rows = torch.randn(42, 20, 128, device="cuda").bfloat16()
    q, k, v = rows.split([16, 2, 2], 1)
    pos = torch.cat([torch.arange(t - n, t) for n, t in zip(news, lens)]).int().cuda()
    slots = torch.cat([st["tables"][b, torch.arange(t - n, t, device="cuda") // 16] * 16
                       + torch.arange(t - n, t, device="cuda") % 16 for b, (n, t) in enumerate(zip(news, lens))]).int()

    def step():
        x = cache.append(rope, q, k, v, pos, slots)
        return cache.attention(x, st["starts"], st["tables"], st["lens"])
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    rows.copy_(torch.randn(42, 20, 128, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    first = out.clone()
    assert torch.equal(first, step())
    x, _ = _kv.turned(q, pos, 128, 1e4, False)
    want, size = _kv.attention(x.bfloat16(), st["k"], st["v"], news, lens, st["tables"])
    # the rotated rows differ from the kernel's by a rounding where they lie next to a border
    assert float((first.double() - want).norm() / want.norm()) < 2.0 ** -7
    cache.check()


def test_lengths_may_change_between_replays():
    """A captured call reads its lengths, starts, tables and groups when it runs."""
    news, lens = [1, 9, 1], [3000, 700, 40]
    st = _kv.batch(news, lens, 2, 128, seed=31, hq=16, junk=False)
    cache = kv().PagedCache.from_pools(st["k"], st["v"])
    groups = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    common = torch.zeros(2, dtype=torch.int32, device="cuda")

    def both():
        return (cache.attention(st["q"], st["starts"], st["tables"], st["lens"]),
                cache.shared_attention(st["q"], st["starts"], st["tables"], st["lens"], groups, common))
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for lens2, news2, prefix in (([2999, 650, 33], [4, 0, 7], [2992, 0]), ([17, 9, 1], [1, 9, 1], [16, 0]),
                                 ([0, 700, 40], [0, 9, 2], [0, 16])):
        st["lens"].copy_(torch.tensor(lens2))
        st["starts"].copy_(torch.tensor([0, *torch.tensor(news2).cumsum(0).tolist()]))
        common.copy_(torch.tensor(prefix))
        st["tables"][2, 0] = st["tables"][1, 0]
        graph.replay()
        torch.cuda.synchronize()
        cache.check()
        n = sum(news2)
        want, size = _kv.attention(st["q"][:n], st["k"], st["v"], news2, lens2, st["tables"])
        for got in out:
            assert _kv.attention_off(got[:n], want, size) <= 1


def test_two_calls_at_once():
    a = _kv.batch([300, 1], [2000, 9000], 2, 128, seed=41, hq=16)
    b = _kv.batch([1, 1, 64], [5000, 70, 64], 4, 64, seed=42, hq=8)
    first = [run(a), run(b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    caches = [kv().PagedCache.from_pools(x["k"], x["v"]) for x in (a, b)]
    got = [[], []]
    for _ in range(20):
        for i, x in enumerate((a, b)):
            got[i].append(caches[i].attention(x["q"], x["starts"], x["tables"], x["lens"], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, first[i]) for y in got[i])


def test_refusals():
    m = kv()
    st = _kv.batch([2], [40], 2, 64, seed=1, hq=4)
    c = m.PagedCache.from_pools(st["k"], st["v"])
    q, s, t, n = st["q"], st["starts"], st["tables"], st["lens"]
    rope = m.Rope(64, 1e4)
    pos = torch.arange(2, device="cuda").int()
    for args in ((q.float(), s, t, n), (q[0], s, t, n), (q[..., :32], s, t, n), (q.cpu(), s, t, n), (q, s[:1], t, n),
                 (q, s.long(), t, n), (q, s, t.long(), n), (q, s, t[0], n), (q, s, t, n.float()), (q, s, t.cpu(), n),
                 (q, s, t, torch.cat([n, n]))):
        with pytest.raises(ValueError):
            c.attention(*args)
    for out in (q.float(), q[:1], torch.empty(2, 8, 64, dtype=q.dtype, device="cuda")[:, ::2], q.cpu()):
        with pytest.raises(ValueError):
            c.attention(q, s, t, n, out=out)
    g = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    p = torch.zeros(1, dtype=torch.int32, device="cuda")
    for args in ((g[:1], p), (g, p[:0]), (g.long(), p), (g, p.cpu())):
        with pytest.raises(ValueError):
            c.shared_attention(q, s, t, n, *args)
    from persistent_moe_decode_gb300 import mk
    for scale in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(mk.MkError):
            c.attention(q, s, t, n, scale=scale)
    with pytest.raises(mk.MkError):
        c.attention(q[:, :3], s, t, n)                       # query heads no multiple of the KV heads
    k = q[:, :2]
    for args in ((q.half(), k.half(), pos), (q, k.float(), pos), (q, k[:1], pos), (q, k, pos[:1]), (q, k, pos.long()),
                 (q[..., :32], k[..., :32], pos), (q.cpu(), k.cpu(), pos)):
        with pytest.raises(ValueError):
            rope.apply(*args)
    with pytest.raises(ValueError):
        rope.apply(q, k, pos, out=(q.float(), k))
    with pytest.raises(mk.MkError):
        rope.apply(q, k, pos, out=(q[:1].expand(2, 4, 64), k))      # rows of one place
    slots = pos.clone()
    for args in ((m.Rope(128, 1e4), q, k, k, pos, slots), (rope, q, q, q, pos, slots), (rope, q, k, k.float(), pos, slots),
                 (rope, q, k, k, pos, slots[:1]), (rope, q, k, k, pos, slots.cpu())):
        with pytest.raises(ValueError):
            c.append(*args)
    with pytest.raises(ValueError):
        c.append(rope, q, k, k, pos, slots, out=q.float())


def test_a_prompt_filled_here_decodes_like_the_oracle():
    """A prompt through the tiny model: dense products by torch, rotary rows, cache rows and attention by these calls;
    the decode step goes on from the pools, against the oracle that saw every token one after the other."""
    import numpy as np

    import oracle
    from persistent_moe_decode_gb300.configs import TINY
    from persistent_moe_decode_gb300.mk import Decoder
    from persistent_moe_decode_gb300.synth import bf16_bits, make_model
    m, d, n = kv(), TINY, 50
    model = make_model(d, 0, "cuda")
    pages, order = 8, [5, 2, 7, 0]
    pools = torch.zeros(2, d.n_layers, pages, d.n_kv_heads, 16, d.head_dim, dtype=torch.bfloat16, device="cuda")
    tokens = torch.randint(0, d.vocab, (n + 1,), generator=torch.Generator().manual_seed(4))
    table = torch.tensor([order], dtype=torch.int32, device="cuda")
    pos = torch.arange(n, device="cuda").int()
    slots = (table[0, (pos // 16).long()] * 16 + pos % 16).int()
    rope = m.Rope(d.head_dim, d.rope_theta)
    h = model.embed[tokens[:n].cuda()].float()

    def norm(x, g):
        return x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + d.rms_eps) * g.float()
    for l in range(d.n_layers):
        x = norm(h, model.attn_norm[l])
        qkv = (x @ model.w_qkv[l].float().T).view(n, -1, d.head_dim)
        q, k, v = qkv.split([d.n_q_heads, d.n_kv_heads, d.n_kv_heads], 1)
        cache = m.PagedCache.from_pools(pools[0, l], pools[1, l])
        q = cache.append(rope, q, k, v, pos, slots)
        o = cache.attention(q, torch.tensor([0, n], device="cuda").int(), table, torch.tensor([n], device="cuda").int())
        cache.check()
        attn = o.float().flatten(1) @ model.w_o[l].float().T
        w, idx = torch.softmax(x @ model.w_router[l].float().T, -1).topk(d.top_k)
        w = w / w.sum(-1, keepdim=True)
        moe = torch.zeros_like(h)
        for e in range(d.n_experts):
            y = (torch.nn.functional.silu(x @ model.w_gate[l, e].float().T) * (x @ model.w_up[l, e].float().T)) \
                @ model.w_down[l, e].float().T
            moe += y * (w * (idx == e)).sum(-1, keepdim=True)
        h = h + attn + moe
    dec = Decoder(model, pools[0], pools[1], 1, len(order))
    logits = torch.zeros(1, d.vocab, device="cuda")
    pt = np.array([order], dtype=np.int32)
    dec.schedule(np.array([int(tokens[n])], dtype=np.int32), pt, np.array([n], dtype=np.int32))
    dec.decode(logits)
    torch.cuda.synchronize()
    assert dec.status()[0] == 0
    got = logits.double().cpu().numpy()
    dec.close()
    oracle.build()
    weights = {x: bf16_bits(getattr(model, x).cpu().contiguous())
               for x in ("embed", "lm_head", "final_norm", "attn_norm", "w_qkv", "w_o", "w_router", "w_gate", "w_up",
                         "w_down")}
    zero = np.zeros(tuple(pools.shape[1:]), dtype=np.uint16)
    orc = oracle.Oracle(dict(d.__dict__), weights, zero.copy(), zero.copy())
    for t in range(n + 1):
        ref = orc.decode_step(np.array([int(tokens[t])], dtype=np.int32), np.array([t], dtype=np.int32), pt, flags=0)
    assert np.abs(got - ref).max() <= 2e-2
    assert np.linalg.norm(got - ref) / np.linalg.norm(ref) <= 1e-2
    assert got.argmax() == ref.argmax()
