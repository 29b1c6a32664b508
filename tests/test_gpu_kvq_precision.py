"""The precision of the 4-bit cache's attention: fp32 calls keep 22 bits of
query and weights (a bound that a call with 11 fails), and contexts of 262,144
tokens, where the mean over the tokens is far smaller than its terms."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from tests import _kvq, _kvq_fp32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from persistent_moe_decode_gb300 import build
    build.build()


@pytest.mark.parametrize("spare", [0, 5000], ids=["cluster", "two kernels"])
@pytest.mark.parametrize("size", [1.0, 8.0])
@pytest.mark.parametrize("n", [5, 16, 100])
@pytest.mark.parametrize("d", [64, 128])
def test_fp32_calls_keep_22_bits_of_query_and_weights(d, n, size, spare):
    """Every dim of a group meets the queries' one element, every token and dim the weights."""
    from persistent_moe_decode_gb300.kvq import QuantCache
    rng = np.random.default_rng(n + d)
    hkv, heads, batch = 2, 8, 8
    pages = -(-n // 16)
    pool = rng.integers(0, 256, size=(pages, hkv * 18 * d), dtype=np.uint8)
    k, v = (rng.normal(size=(n, hkv, d)).astype(np.float32).astype(np.float64) for _ in range(2))
    _kvq.store(pool, hkv, d, k, v, np.arange(n))
    keys, values = _kvq.load(pool, hkv, d, np.arange(n))
    q = _kvq_fp32.queries(rng, batch, hkv * heads, d, size)
    c = QuantCache.from_pool(torch.from_numpy(pool).cuda(), hkv, d)
    table = torch.full((batch, pages + spare), -1, dtype=torch.int32, device="cuda")
    table[:, :pages] = torch.arange(pages, dtype=torch.int32, device="cuda")
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    got = c.attention(torch.from_numpy(q).float().cuda(), table, lens).double().cpu().numpy()
    c.check()
    for b in range(batch):
        for g in range(hkv):
            h = slice(g * heads, g * heads + heads)
            out, S, P, E = _kvq_fp32.exact(q[b, h], *([a[:, g] for a in x] for x in (keys, values)), d ** -0.5)
            err = np.abs(got[b, h] - out) / _kvq_fp32.tolerance(out, S, P, E, n)
            assert (err <= 1).all(), (b, g, float(err.max()))


@pytest.mark.parametrize("batch", [1, 32])
@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (128, torch.float32), (64, torch.float32)])
def test_attention_over_262144_tokens(d, dtype, batch):
    """One sequence, and 32 over the same pages (hundreds of pages a warp), against 64 bits, by the norm of the error
    relative to the norm of the results.  Per element, with p the softmax, C = sqrt(sum (p step (code - 8))^2) and
    V = sqrt(sum (p value)^2), what sums of independent signs come to:
      the result's rounding: half a step;
      weights: 2^-11 (BF16) or 2^-22 of each term, the rms a factor sqrt(3) less, against C;
      scores: a group's sum takes 4 matrix products a half, each loses at most 2^-23 (fp32, codes - 8) or, of
        subnormal codes, 2^-24 of 2 (BF16; the query scaled to 2^13) for each of 17 addends; 8 fp32 roundings of T;
        ln 2 of that, and 2^-22 of ex2, against V; six times each of these rms values;
      sums: a page's addition loses 2^-24 (fp32) or, in the matrix product, 17 2^-23 (BF16) of the running sum, which
        is sqrt(tokens so far / n) of C, twice that at most; fp32 page sums 17 2^-23 of their largest terms, 2 / sqrt(n) of C."""
    from persistent_moe_decode_gb300.kvq import QuantCache
    n, heads, f32 = 262144, 8, dtype == torch.float32
    gen = torch.Generator("cuda").manual_seed(d + batch)
    c = QuantCache(n // 16, 1, d)
    k = torch.randn(n, 1, d, device="cuda", generator=gen)
    v = torch.randn(n, 1, d, device="cuda", generator=gen) * 0.5
    table = torch.randperm(n // 16, device="cuda", generator=gen).int()
    t = torch.arange(n, device="cuda")
    slots = (table[t // 16] * 16 + t % 16).int()
    c.write(k, v, slots)
    lens = n - 1000 * np.arange(batch)
    q = torch.randn(batch, heads, d, device="cuda", generator=gen).to(dtype)
    got = c.attention(q, table[None].repeat(batch, 1), torch.from_numpy(lens).int().cuda())
    c.check()
    got, pool, slots = got.double().cpu().numpy().reshape(-1, d), c.pool.cpu().numpy(), slots.cpu().numpy()
    qh = q.double().cpu().numpy().reshape(-1, d)
    last = np.repeat(lens, heads)
    unit = math.log2(math.e) / math.sqrt(d)
    m, den = np.full(len(qh), -np.inf), np.zeros(len(qh))
    num, C2, V2 = (np.zeros((len(qh), d)) for _ in range(3))
    T, top_step = np.zeros(len(qh)), 0.0
    for i in range(0, n, 16384):
        (kc, ks, kl), (vc, vs, vl) = (tuple(a[:, 0] for a in x) for x in _kvq.load(pool, 1, d, slots[i:i + 16384]))
        x = unit * (qh @ (ks * kc + kl).T)
        x[np.arange(i, i + 16384)[None] >= last[:, None]] = -np.inf
        T = np.maximum(T, unit * (np.abs(qh) @ (ks * np.abs(kc - 8) + np.abs(kl + 8 * ks)).T).max(1))
        top_step = max(top_step, ks.max())
        new = np.maximum(m, x.max(1))
        keep, p = np.exp2(m - new), np.exp2(x - new[:, None])
        m, den = new, den * keep + p.sum(1)
        num = num * keep[:, None] + p @ (vs * vc + vl)
        C2 = C2 * keep[:, None] ** 2 + (p * p) @ (vs * (vc - 8)) ** 2
        V2 = V2 * keep[:, None] ** 2 + (p * p) @ (vs * vc + vl) ** 2
    out, C, V = num / den[:, None], np.sqrt(C2) / den[:, None], np.sqrt(V2) / den[:, None]
    top_q = np.abs(qh).max(1)
    group = 4 * 17 * unit * top_step * top_q * (8 * 2.0 ** -23 if f32 else 2.0 ** -13)
    score = (d // 64) * group + 8 * 2.0 ** -24 * T
    weight = (2.0 ** -22 if f32 else 2.0 ** -11) / math.sqrt(3)
    terms = 6 * np.sqrt((weight * C) ** 2 + ((math.log(2) * score + 2.0 ** -22)[:, None] * V) ** 2)
    pages, warps = n / 16, 8 * (152 if f32 and d == 128 else 304)
    a_warp = batch * pages / warps + 8
    sums = 2 * pages * math.sqrt(16 * a_warp / n) * (2.0 ** -24 if f32 else 17 * 2.0 ** -23)
    sums += pages * 17 * 2.0 ** -23 * 2 / math.sqrt(n) if f32 else 0
    norm = np.linalg.norm
    bound = (2.0 ** -24 if f32 else 2.0 ** -8) * norm(out) + norm(terms) + sums * norm(C)
    err = norm(got - out)
    print(f"d {d} {dtype} batch {batch}: relative error {err / norm(out):.2e}, bound {bound / norm(out):.2e}")
    assert bound <= (1e-3 if f32 else 0.04) * norm(out)      # codes 0 .. 15 in place of code - 8 would be 0.08 off
    assert err <= bound


# ------------------------------------------------ the number range include/mk.h gives

LIMITS = {
    "query 2^79": dict(q=2.0 ** 77, k=2.0 ** -76),
    "keys 2^79": dict(q=2.0 ** -76, k=2.0 ** 77),
    "values 2^79": dict(v=2.0 ** 77),
    "all": dict(q=2.0 ** -78, k=2.0 ** 77, v=2.0 ** 77),
    "scale 2^20": dict(q=2.0 ** -19, scale=2.0 ** 16),
    "small": dict(q=2.0 ** -100, k=2.0 ** 70, v=2.0 ** -100, scale=2.0 ** 20),
}


def range_case(rng, d, n, dtype, q=1.0, k=1.0, v=1.0):
    hkv, heads, batch = 1, 8, 2
    pages = -(-n // 16)
    pool = rng.integers(0, 256, size=(pages, hkv * 18 * d), dtype=np.uint8)
    kr, vr = (rng.normal(size=(n, hkv, d)).clip(-4, 4).astype(np.float32).astype(np.float64) for _ in range(2))
    _kvq.store(pool, hkv, d, kr * k, vr * v, np.arange(n))
    qr = torch.from_numpy(rng.normal(size=(batch, hkv * heads, d)).clip(-4, 4) * q).float().to(dtype)
    return pool, np.arange(pages, dtype=np.int32)[None].repeat(batch, 0), qr


def over(pool, table, q, n, **kw):
    from persistent_moe_decode_gb300.kvq import QuantCache
    c = QuantCache.from_pool(torch.from_numpy(pool).cuda(), 1, q.shape[-1])
    out = c.attention(q.cuda(), torch.from_numpy(table).cuda(), torch.full((len(table),), n, dtype=torch.int32,
                                                                          device="cuda"), **kw)
    c.check()
    return out.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("name", LIMITS)
@pytest.mark.parametrize("d", [64, 128])
def test_attention_at_the_ends_of_the_number_range(d, name, dtype):
    rng = np.random.default_rng(d)
    kw, n = dict(LIMITS[name]), 500
    scale = kw.pop("scale", d ** -0.5)
    pool, table, q = range_case(rng, d, n, dtype, **kw)
    got = over(pool, table, q, n, scale=scale)
    keys, values = _kvq.load(pool, 1, d, np.arange(n))
    for b in range(len(table)):
        ref, spread, score = _kvq.attention(q[b].double().numpy(), keys, values, 1, scale)
        tol = _kvq.attention_tolerance(ref, spread, score, n, d, dtype == torch.float32)
        assert (np.abs(got[b] - ref) <= tol).all(), float((np.abs(got[b] - ref) / tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes", [(2.0 ** 50, 2.0 ** 44), (2.0 ** 17, 2.0 ** 77), (2.0 ** 77, 2.0 ** 17)])
def test_scores_near_2_to_the_100_leave_the_largest_token(sizes, dtype):
    """The gap between the two largest scores is far above their error, so all weight is one token's."""
    rng = np.random.default_rng(16)
    d, n = 128, 300
    pool, table, q = range_case(rng, d, n, dtype, q=sizes[0], k=sizes[1])
    got = over(pool, table, q, n)
    keys, values = _kvq.load(pool, 1, d, np.arange(n))
    for b in range(len(table)):
        qb = q[b].double().numpy()
        kx = (keys[1] * keys[0] + keys[2])[:, 0]
        bound = np.abs(qb).sum(1).max() * np.abs(kx).max() * d ** -0.5
        assert 2.0 ** 99 < bound < 2.0 ** 100
        x = np.sort(qb @ kx.T * d ** -0.5, 1)
        assert (x[:, -1] - x[:, -2] > 2.0 ** -9 * bound).all()
        ref, spread, _ = _kvq.attention(qb, keys, values, 1, d ** -0.5)
        tol = _kvq.attention_tolerance(ref, spread, np.zeros(len(qb)), n, d, dtype == torch.float32)
        assert (np.abs(got[b] - ref) <= tol).all()
