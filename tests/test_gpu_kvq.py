"""The 4-bit KV cache operators (mk_kvq_*, QuantCache) against a restatement
in 64 bits (tests/_kvq.py): stored bytes and read-back values equal, attention
within the tolerance its roundings give."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from tests import _kvq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from persistent_moe_decode_gb300 import build
    build.build()


def QuantCache(*a, **kw):
    from persistent_moe_decode_gb300.kvq import QuantCache as Q
    return Q(*a, **kw)


def random_pool(rng, pages, hkv, d):
    """Random bytes: what no row was written to may hold anything."""
    return rng.integers(0, 256, size=(pages, hkv * 18 * d), dtype=np.uint8)


def cache_over(pool, hkv, d):
    from persistent_moe_decode_gb300.kvq import QuantCache as Q
    return Q.from_pool(torch.from_numpy(pool.copy()).cuda(), hkv, d)


def to_dtype(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).float().to(dtype)


def host(t):
    return t.double().cpu().numpy()


def kv_rows(rng, n, hkv, d, dtype):
    off = rng.normal(size=(hkv, d)) * (rng.random((hkv, d)) < 0.06) * 4
    k = to_dtype(rng.normal(size=(n, hkv, d)) + off, dtype)
    v = to_dtype(rng.normal(size=(n, hkv, d)) * 0.5, dtype)
    return k, v


# ------------------------------------------------------------- store and read

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,hkv", [(1, 1), (7, 3), (16, 4), (33, 2), (200, 8)])
def test_write_leaves_the_defined_bytes_and_read_gives_their_values(n, hkv, d, dtype):
    rng = np.random.default_rng(n * 1000 + hkv * 10 + d)
    pages = n // 16 + 3
    pool = random_pool(rng, pages, hkv, d)
    c = cache_over(pool, hkv, d)
    k, v = kv_rows(rng, n, hkv, d, dtype)
    slots = rng.permutation(pages * 16)[:n].astype(np.int32)
    slots[::5] = -1
    c.write(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    _kvq.store(pool, hkv, d, host(k), host(v), slots)
    assert np.array_equal(c.pool.cpu().numpy(), pool)          # rows that were not written included
    live = slots >= 0
    keys, values = _kvq.load(pool, hkv, d, np.maximum(slots, 0))
    for dt in (torch.bfloat16, torch.float32):
        got = c.read(torch.from_numpy(slots).cuda(), dt)
        for g, (code, step, low) in zip(got, (keys, values)):
            want = torch.from_numpy(np.where(live[:, None, None], step * code + low, 0.0)).float().to(dt)
            assert torch.equal(g.cpu(), want)
    c.check()


@pytest.mark.parametrize("d", [64, 128])
def test_write_at_the_edges_of_the_number_range(d):
    """Constant groups, signed zeros, subnormals, the largest numbers, ties, NaN and infinities."""
    rng = np.random.default_rng(d)
    f = np.float32
    rows = [np.zeros(64), np.full(64, -3.5), np.where(np.arange(64) % 2, 0.0, -0.0),
            np.arange(64) % 16 * 1.0, np.arange(64) / 2.0 % 15.5, -np.arange(64) / 8.0,
            rng.normal(size=64) * 1e-39, rng.normal(size=64) * 1e-44, rng.normal(size=64) * 1e37,
            np.where(np.arange(64) == 3, 3.3e38, -1.0), np.where(np.arange(64) % 2, 3.3e38, -3.3e38),
            np.where(np.arange(64) == 5, np.nan, 1.0), np.where(np.arange(64) == 5, np.inf, 1.0),
            np.where(np.arange(64) == 5, -np.inf, 1.0), np.full(64, np.finfo(f).min),
            1.0 + np.arange(64) * 2.0 ** -23, 1e-20 * np.arange(64) - (np.arange(64) == 9),
            np.arange(64) % 31 * 0.5 + 2.0 ** -20 * rng.integers(-2, 3, size=64) - 7.5]
    rows += [rng.normal(size=64) * 10.0 ** rng.uniform(-30, 30) for _ in range(200)]
    # around every half-way point of a step of 1: the neighbours of k + 1/2 - 7.5
    ties = np.arange(15) + 0.5
    near = np.concatenate([np.nextafter(f(ties), f(0)), f(ties), np.nextafter(f(ties), f(99)), [0, 15] * 9, [0]])
    rows.append(near[:64])
    x = np.array(rows, dtype=np.float32)
    while len(x) % (2 * (d // 64)):
        x = np.concatenate([x, x[:1]])
    for dtype in (torch.float32, torch.bfloat16):
        t = torch.from_numpy(x).to(dtype).reshape(2, -1, 1, d)
        n = t.shape[1]
        pool = random_pool(rng, n // 16 + 1, 1, d)
        c = cache_over(pool, 1, d)
        slots = np.arange(n, dtype=np.int32)
        c.write(t[0].cuda(), t[1].cuda(), torch.from_numpy(slots).cuda())
        _kvq.store(pool, 1, d, host(t[0]), host(t[1]), slots)
        assert np.array_equal(c.pool.cpu().numpy(), pool)
        got = c.read(torch.from_numpy(slots).cuda(), torch.float32)
        for g, x0, (code, step, low) in zip(got, t, _kvq.load(pool, 1, d, slots)):
            want = torch.from_numpy(step * code + low).float()
            assert torch.equal(g.cpu().isnan(), want.isnan())
            assert torch.equal(g.cpu().nan_to_num(7.0), want.nan_to_num(7.0))
            # the promise to the user: half a step, and a constant group comes back as it was (to BF16)
            ok = np.isfinite(step * code + low)
            err = np.abs(host(g) - host(x0))
            assert (err[ok] <= (0.5 * step + 2.0 ** -7 * np.abs(low) * (step == 0) + 2.0 ** -23 * np.abs(host(x0)))[ok]).all()


def test_write_of_strided_rows_and_read_beside_other_rows():
    """Keys and values as slices of a fused QKV row, rows behind the call's left alone."""
    rng = np.random.default_rng(5)
    hkv, d, n = 2, 128, 21
    qkv = to_dtype(rng.normal(size=(n, (4 + 2 * hkv) * d)), torch.float32).cuda()
    k = qkv[:, 4 * d:(4 + hkv) * d].unflatten(1, (hkv, d))
    v = qkv[:, (4 + hkv) * d:].unflatten(1, (hkv, d))
    pool = random_pool(rng, 4, hkv, d)
    c = cache_over(pool, hkv, d)
    slots = np.arange(9, 9 + n, dtype=np.int32)
    c.write(k, v, torch.from_numpy(slots).cuda())
    _kvq.store(pool, hkv, d, host(k), host(v), slots)
    assert np.array_equal(c.pool.cpu().numpy(), pool)
    # transposed and unaligned sources go through a copy
    kt = k.transpose(0, 1).contiguous().transpose(0, 1)
    odd = torch.empty(n * hkv * d + 1, device="cuda")[1:].view(n, hkv, d).copy_(v)
    c2 = cache_over(np.zeros_like(pool), hkv, d)
    c2.write(kt, odd, torch.from_numpy(slots).cuda())
    assert all(torch.equal(a, b) for a, b in zip(c2.read(torch.from_numpy(slots).cuda()),
                                                 c.read(torch.from_numpy(slots).cuda())))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hkv,d,n", [(1, 64, 1), (4, 128, 5), (3, 64, 37), (8, 128, 11)])
def test_pages_convert_and_return(hkv, d, n, dtype):
    rng = np.random.default_rng(hkv + d + n)
    pages = n + 4
    pool = random_pool(rng, pages, hkv, d)
    c = cache_over(pool, hkv, d)
    kp, vp = (to_dtype(rng.normal(size=(pages + 1, hkv, 16, d)), dtype) for _ in range(2))
    src, dst = rng.permutation(pages + 1)[:n].astype(np.int32), rng.permutation(pages)[:n].astype(np.int32)
    if n > 4:
        src[1], dst[3] = -1, -1
    c.write_pages(kp.cuda(), vp.cuda(), torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda())
    live = (src >= 0) & (dst >= 0)
    rows = [host(x)[src[live]].transpose(0, 2, 1, 3).reshape(-1, hkv, d) for x in (kp, vp)]
    slots = (dst[live][:, None] * 16 + np.arange(16)).reshape(-1)
    _kvq.store(pool, hkv, d, *rows, slots)
    assert np.array_equal(c.pool.cpu().numpy(), pool)
    # and back: untouched pages keep their content, a negative source gives zeros
    ko, vo = (torch.full((pages, hkv, 16, d), 5.0, dtype=dtype, device="cuda") for _ in range(2))
    back = rng.permutation(pages)[:n].astype(np.int32)
    frm = dst.copy()
    if n > 4:
        back[0] = -1
    c.read_pages(torch.from_numpy(frm).cuda(), ko, vo, torch.from_numpy(back).cuda())
    want = [np.full((pages, hkv, 16, d), 5.0) for _ in range(2)]
    for i in range(n):
        if back[i] < 0:
            continue
        for w, (code, step, low) in zip(want, _kvq.load(pool, hkv, d, max(frm[i], 0) * 16 + np.arange(16))):
            val = np.zeros((16, hkv, d)) if frm[i] < 0 else step * code + low
            w[back[i]] = val.transpose(1, 0, 2)
    for g, w in zip((ko, vo), want):
        w = torch.from_numpy(w).float().to(dtype)
        assert torch.equal(g.cpu().nan_to_num(7.0), w.nan_to_num(7.0))
    c.check()


# ----------------------------------------------------------------- attention

def attention_case(rng, hkv, grp, d, lens, dtype, spare=1, pool=None, kmul=1.0, vmul=None, qmul=1.0):
    """A cache of the given lengths on permuted pages of garbage, its page tables and queries."""
    need = [-(-n // 16) for n in lens]
    pages = sum(need) + 2
    pool = random_pool(rng, pages, hkv, d)
    table = np.full((len(lens), max(need) + spare), -7, dtype=np.int32)
    table[:, :] = rng.choice([-1, 1 << 30, pages], size=table.shape)   # entries past a sequence are not read
    perm = rng.permutation(pages)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        if n:
            t = np.arange(n)
            k, v = kv_rows(rng, n, hkv, d, torch.bfloat16)
            k, v = host(k) * kmul, host(v)
            if vmul is not None:
                v = v * vmul(t)[:, None, None]
            k, v = host(to_dtype(k, torch.float32)), host(to_dtype(v, torch.float32))
            _kvq.store(pool, hkv, d, k, v, table[b, t // 16] * 16 + t % 16)
    q = to_dtype(rng.normal(size=(len(lens), hkv * grp, d)) * qmul, dtype)
    return pool, table, q


def check_attention(out, pool, table, q, lens, hkv, scale=None):
    d, f32 = q.shape[-1], q.dtype == torch.float32
    scale = 1 / math.sqrt(d) if scale is None else scale
    got = host(out)
    for b, n in enumerate(lens):
        t = np.arange(n)
        keys, values = _kvq.load(pool, hkv, d, table[b, t // 16] * 16 + t % 16)
        ref, spread, score = _kvq.attention(host(q)[b], keys, values, hkv, scale)
        tol = _kvq.attention_tolerance(ref, spread, score, n, d, f32)
        err = np.abs(got[b] - ref)
        assert (err <= tol).all(), (b, n, float((err / tol).max()), float(err.max()))


def run_attention(pool, table, q, lens, hkv, **kw):
    c = cache_over(pool, hkv, q.shape[-1])
    out = c.attention(q.cuda(), torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                      **kw)
    c.check()
    return out


LENS = [[1], [16], [17, 0, 1], [15, 16, 31, 33, 128, 129], [700], [0, 0], [5, 2000, 64, 0, 1023]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,grp", [(1, 1), (2, 2), (4, 8), (3, 5)])
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
def test_attention(lens, hkv, grp, d, dtype):
    rng = np.random.default_rng(hkv * 100 + grp * 10 + d + sum(lens))
    pool, table, q = attention_case(rng, hkv, grp, d, lens, dtype)
    check_attention(run_attention(pool, table, q, lens, hkv), pool, table, q, lens, hkv)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hkv,grp,d,lens", [(1, 16, 128, [100, 1]), (2, 9, 64, [333]), (1, 71, 128, [40]),
                                            (40, 1, 64, [50, 3])])
def test_attention_of_many_heads(hkv, grp, d, lens, dtype):
    rng = np.random.default_rng(grp)
    pool, table, q = attention_case(rng, hkv, grp, d, lens, dtype)
    check_attention(run_attention(pool, table, q, lens, hkv), pool, table, q, lens, hkv)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hkv,grp,d,lens", [(1, 8, 128, [20000]), (4, 4, 64, [12345, 1, 7000]),
                                            (2, 8, 128, [9000] * 3 + [0] + [40] * 20)])
def test_attention_of_long_and_uneven_contexts(hkv, grp, d, lens, dtype):
    rng = np.random.default_rng(len(lens))
    pool, table, q = attention_case(rng, hkv, grp, d, lens, dtype, spare=0)
    check_attention(run_attention(pool, table, q, lens, hkv), pool, table, q, lens, hkv)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spare", [40, 300, 3001])
@pytest.mark.parametrize("lens", [[1], [17, 0, 1], [700, 128, 129, 0], [0, 0], [5, 2000, 64, 0, 1023], [16] * 70],
                         ids=lambda x: "-".join(map(str, x[:5])))
def test_attention_with_wide_page_tables(lens, spare, d, dtype):
    """Room for far longer sequences than there are: every way of cutting the pages, at every length."""
    rng = np.random.default_rng(spare + d)
    pool, table, q = attention_case(rng, 2, 4, d, lens, dtype, spare=spare)
    check_attention(run_attention(pool, table, q, lens, 2), pool, table, q, lens, 2)


@pytest.mark.parametrize("batch,n", [(300, 40), (700, 0), (1500, 20)])
def test_attention_of_a_large_batch(batch, n):
    """More sequences than one window of the plan, idle ones and one long one among them."""
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, n + 1, size=batch)
    lens[rng.random(batch) < 0.2] = 0
    lens[batch // 2 + 7] = 3000
    pool, table, q = attention_case(rng, 1, 2, 64, [int(x) for x in lens], torch.bfloat16)
    check_attention(run_attention(pool, table, q, [int(x) for x in lens], 1), pool, table, q, lens, 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kw", [
    dict(qmul=30.0),                                                # one key takes nearly all
    dict(qmul=1e-3),                                                # nearly uniform weights
    dict(qmul=0.0),                                                 # uniform weights
    dict(qmul=1e18, kmul=1e-18), dict(qmul=1e-30, kmul=1e25),       # far from FP16's range
    dict(vmul=lambda t: np.where(t == 3, 2.0 ** 40, 1.0)),          # one value far larger
    dict(vmul=lambda t: np.exp2(-(t % 60.0))),                      # steps over 60 powers of two
    dict(vmul=lambda t: np.exp2(t / 16 % 90.0 - 45)),               # growing from page to page
    dict(vmul=lambda t: np.zeros_like(t, dtype=float)),             # steps of 0
], ids=["peaked", "flat", "uniform", "largeq", "smallq", "outlier", "spread", "growing", "zeros"])
def test_attention_over_unusual_scales(kw, dtype):
    rng = np.random.default_rng(11)
    lens = [300, 17, 1000]
    pool, table, q = attention_case(rng, 2, 4, 128, lens, dtype, **kw)
    check_attention(run_attention(pool, table, q, lens, 2), pool, table, q, lens, 2)


def test_attention_scores_that_grow_and_fall():
    """The running references move page by page: keys ever closer to, then ever farther from, the query."""
    rng = np.random.default_rng(3)
    d, hkv, n = 128, 1, 800
    q = to_dtype(rng.normal(size=(1, 4, d)), torch.bfloat16)
    for sign in (1, -1):
        amount = np.linspace(-6, 6, n) * sign
        k = rng.normal(size=(n, 1, d)) * 0.1 + amount[:, None, None] * host(q)[0, 0]
        v = rng.normal(size=(n, 1, d))
        pool = random_pool(rng, n // 16 + 1, hkv, d)
        slots = np.arange(n)
        _kvq.store(pool, hkv, d, host(to_dtype(k, torch.float32)), host(to_dtype(v, torch.float32)), slots)
        table = np.arange(n // 16 + 1, dtype=np.int32)[None]
        check_attention(run_attention(pool, table, q, [n], hkv), pool, table, q, [n], hkv)


def test_attention_scale_strides_and_output_rows():
    rng = np.random.default_rng(8)
    hkv, grp, d, lens = 2, 4, 128, [70, 300, 9]
    pool, table, q = attention_case(rng, hkv, grp, d, lens, torch.bfloat16)
    c = cache_over(pool, hkv, d)
    wide = torch.zeros(3, 8 + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")   # q in a fused QKV row
    wide[:, :8] = q.cuda()
    tb, ln = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full((5, 8, d), 3.0, dtype=torch.bfloat16, device="cuda")
    got = c.attention(wide[:, :8], tb, ln, scale=0.3, out=out[1:4])
    assert got.data_ptr() == out[1:4].data_ptr() and (out[[0, 4]] == 3).all()
    check_attention(got, pool, table, q, lens, hkv, scale=0.3)
    # a transposed query and a column-sliced table go through a copy
    again = c.attention(q.cuda().transpose(0, 1).contiguous().transpose(0, 1),
                        torch.cat([tb, tb], 1)[:, :tb.shape[1]], ln, scale=0.3)
    assert torch.equal(again, got)
    # the output over the query itself
    same = q.cuda()
    c.attention(same, tb, ln, scale=0.3, out=same)
    assert torch.equal(same, got)
    # a workspace that is missing, short or misaligned is refused; short page tables need none
    from persistent_moe_decode_gb300 import mk
    need = mk.mk_kvq_workspace(c._c, mk.MK_TYPE_BF16, 8, 3, 5000)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    args = (c._c, q.cuda().data_ptr(), 8 * d, got.data_ptr(), 8 * d, mk.MK_TYPE_BF16, 8, 3, tb.data_ptr(), 5000,
            ln.data_ptr(), 0.3)
    for ptr, n in ((None, need), (ws.data_ptr(), need - 1), (ws.data_ptr() + 8, need)):
        with pytest.raises(mk.MkError) as e:
            mk.mk_kvq_attention(*args, ptr, n)
        assert e.value.code == mk.MK_ERR_BAD_ARG
    assert need > 0 and mk.mk_kvq_workspace(c._c, mk.MK_TYPE_BF16, 8, 3, tb.shape[1]) == 0
    # nothing to do
    assert c.attention(q.cuda()[:0], tb[:0], ln[:0]).shape == (0, 8, d)
    none = c.attention(q.cuda(), tb[:, :0], torch.zeros_like(ln))
    assert (none == 0).all()
    c.check()


def test_attention_rows_do_not_depend_on_the_batch():
    """A sequence's result is the same alone, in a batch and with idle slots, and from call to call."""
    rng = np.random.default_rng(21)
    hkv, grp, d, lens = 4, 8, 128, [1500, 0, 40, 3001]
    pool, table, q = attention_case(rng, hkv, grp, d, lens, torch.bfloat16)
    first = run_attention(pool, table, q, lens, hkv)
    assert torch.equal(first, run_attention(pool, table, q, lens, hkv))
    for b, n in enumerate(lens):
        alone = run_attention(pool, table[b:b + 1], q[b:b + 1], [n], hkv)
        keys = _kvq.load(pool, hkv, d, table[b, np.arange(n) // 16] * 16 + np.arange(n) % 16)
        ref, spread, score = _kvq.attention(host(q)[b], *keys, hkv, 1 / math.sqrt(d))
        tol = _kvq.attention_tolerance(ref, spread, score, n, d, False)
        assert (np.abs(host(alone)[0] - host(first)[b]) <= 2 * tol).all()


def test_a_nan_in_the_cache_stays_with_its_heads():
    rng = np.random.default_rng(2)
    hkv, grp, d, n = 2, 2, 128, 50
    pool, table, q = attention_case(rng, hkv, grp, d, [n, n], torch.bfloat16)
    c = cache_over(pool, hkv, d)
    slot = torch.tensor([int(table[0, 2]) * 16 + 5], dtype=torch.int32, device="cuda")
    k, v = c.read(slot, torch.float32)
    v[0, 0, 70] = float("inf")                      # KV head 0, dims 64..127 of one value
    c.write(k, v, slot)
    out = c.attention(q.cuda(), torch.from_numpy(table).cuda(),
                      torch.tensor([n, n], dtype=torch.int32, device="cuda")).float().cpu()
    assert out[0, :2, 64:].isnan().all() and not out[0, :2, :64].isnan().any()
    assert not out[0, 2:].isnan().any() and not out[1].isnan().any()


def test_pages_behind_two_gigabytes():
    """Offsets past 31 bits: the last pages of a large pool."""
    hkv, d = 4, 128
    pages = 2 ** 31 // (hkv * 18 * d) + 5000
    rng = np.random.default_rng(1)
    c = QuantCache(pages, hkv, d)
    n = 100
    ids = np.arange(pages - 7, pages, dtype=np.int32)[::-1].copy()
    slots = ids[np.arange(n) // 16] * 16 + np.arange(n, dtype=np.int32) % 16
    k, v = kv_rows(rng, n, hkv, d, torch.bfloat16)
    s = torch.from_numpy(slots).cuda()
    c.write(k.cuda(), v.cuda(), s)
    small = np.zeros((7, hkv * 18 * d), dtype=np.uint8)
    _kvq.store(small, hkv, d, host(k), host(v), slots - (pages - 7) * 16)
    assert np.array_equal(c.pool[-7:].cpu().numpy(), small)
    q = to_dtype(rng.normal(size=(1, 32, d)), torch.bfloat16)
    out = c.attention(q.cuda(), torch.from_numpy(ids[None]).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"))
    check_attention(out, small, ids[None] - (pages - 7), q, [n], hkv)
    kb = c.read(s, torch.float32)[0]
    code, step, low = _kvq.load(small, hkv, d, slots - (pages - 7) * 16)[0]
    assert torch.equal(kb.cpu(), torch.from_numpy(step * code + low).float())
    c.check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hkv,d,n", [(5, 128, 1500), (7, 64, 1100), (1, 128, 8000)])
def test_long_calls_store_the_same_bytes_by_page_and_by_row(hkv, d, n, dtype):
    """Calls long enough for several heads a block, and a last block with fewer: whole pages, and the same rows in
    calls of several lengths, leave the same bytes (those of the restatement on a sample) and read back alike."""
    gen = torch.Generator("cuda").manual_seed(n)
    kp, vp = (torch.randn(n, hkv, 16, d, device="cuda", generator=gen).to(dtype) for _ in range(2))
    a, b = QuantCache(n, hkv, d), QuantCache(n, hkv, d)
    ids = torch.randperm(n, device="cuda", generator=gen).to(torch.int32)
    src = torch.arange(n, dtype=torch.int32, device="cuda")
    ids[n // 3] = -1
    src[n // 2] = -1
    a.write_pages(kp, vp, src, ids)
    kr, vr = (x.transpose(1, 2).reshape(n * 16, hkv, d) for x in (kp, vp))
    dst = torch.where((src < 0) | (ids < 0), -1, ids)
    slots = torch.where(dst[:, None] < 0, -1, dst[:, None] * 16 + torch.arange(16, device="cuda")).reshape(-1).int()
    at = 0
    for m in (1, 3001, 7, 9000, n * 16):
        b.write(kr[at:at + m], vr[at:at + m], slots[at:at + m])
        at += m
    assert at >= n * 16 and torch.equal(a.pool, b.pool)
    some = [0, 1, n // 3, n // 2, n // 2 + 1, n - 2, n - 1]
    for i in some:
        if int(dst[i]) < 0:
            continue
        one = np.zeros((1, hkv * 18 * d), dtype=np.uint8)
        rows = [host(x[i].cpu()).transpose(1, 0, 2) for x in (kp, vp)]
        _kvq.store(one, hkv, d, *rows, np.arange(16))
        assert np.array_equal(a.pool[int(dst[i])].cpu().numpy(), one[0])
    ko, vo = torch.zeros_like(kp), torch.zeros_like(vp)
    a.read_pages(dst, ko, vo, torch.arange(n, dtype=torch.int32, device="cuda"))
    kb, vb = a.read(slots, dtype)
    for x, y in ((ko, kb), (vo, vb)):
        assert torch.equal(x.transpose(1, 2).reshape(n * 16, hkv, d), y)
    a.check()
    b.check()


# -------------------------------------------------- indexes out of range, streams, graphs

def test_bad_indexes_are_flagged_and_touch_nothing():
    from persistent_moe_decode_gb300 import mk
    rng = np.random.default_rng(4)
    hkv, d, pages = 2, 64, 4
    pool = random_pool(rng, pages, hkv, d)
    c = cache_over(pool, hkv, d)
    k, v = kv_rows(rng, 3, hkv, d, torch.bfloat16)
    slots = np.array([5, pages * 16, 2 ** 31 - 1], dtype=np.int32)
    c.write(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    with pytest.raises(mk.MkError) as e:
        c.check()
    assert e.value.code == mk.MK_ERR_BAD_PAGE
    _kvq.store(pool, hkv, d, host(k), host(v), [5, -1, -1])
    assert np.array_equal(c.pool.cpu().numpy(), pool)
    c.check()                                        # the record was cleared
    kp = torch.full((pages, hkv, 16, d), 2.0, dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    idx = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    c.read_pages(idx(0, pages, 1), kp, vp, idx(pages, 1, 2 ** 30))
    assert (kp == 2).all() and (vp == 2).all()
    with pytest.raises(mk.MkError):
        c.check()
    c.write_pages(kp, vp, idx(pages, 0), idx(0, pages))
    assert np.array_equal(c.pool.cpu().numpy(), pool)
    with pytest.raises(mk.MkError):
        c.check()


def test_attention_with_a_bad_page_or_length_gives_nan_rows():
    from persistent_moe_decode_gb300 import mk
    rng = np.random.default_rng(6)
    hkv, grp, d, lens = 2, 4, 128, [40, 600, 16]
    for bad in (-1, 1 << 30):
        pool, table, q = attention_case(rng, hkv, grp, d, lens, torch.bfloat16)
        c = cache_over(pool, hkv, d)
        t = table.copy()
        t[1, 20] = bad
        out = c.attention(q.cuda(), torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
        assert out[1].isnan().all() and not out[[0, 2]].isnan().any()
        with pytest.raises(mk.MkError) as e:
            c.check()
        assert e.value.code == mk.MK_ERR_BAD_PAGE
    for bad in (-5, table.shape[1] * 16 + 1, 2 ** 31 - 1):
        ln = torch.tensor([40, bad, 16], dtype=torch.int32, device="cuda")
        out = c.attention(q.cuda(), torch.from_numpy(table).cuda(), ln)
        assert out[1].isnan().all() and not out[[0, 2]].isnan().any()
        check_attention(out[[0, 2]], pool, table[[0, 2]], q[[0, 2]], [40, 16], hkv)
        with pytest.raises(mk.MkError) as e:
            c.check()
        assert e.value.code == mk.MK_ERR_BAD_ARG


@pytest.mark.parametrize("spare", [1, 5000], ids=["cluster", "workspace"])
def test_calls_on_a_stream_and_captured_graphs_side_by_side(spare):
    """A step of write and attention captured twice over one cache, the two graphs replayed at once on two
    streams with new contents, against plain calls."""
    rng = np.random.default_rng(9)
    hkv, grp, d = 4, 8, 128
    lens = [2000, 5000, 333]
    pool, table, q = attention_case(rng, hkv, grp, d, lens, torch.bfloat16, spare=spare)
    c = cache_over(pool, hkv, d)
    tb = torch.from_numpy(table).cuda()
    sets, graphs = [], []
    for half in range(2):
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda") - 100 * half
        pos = ln.long() - 1
        k, v = kv_rows(rng, 3, hkv, d, torch.bfloat16)
        # the two graphs write rows of their own (the last token each sees)
        slots = (tb[torch.arange(3), pos // 16] * 16 + pos % 16).to(torch.int32)
        sets.append(dict(q=q.cuda() + half, k=k.cuda(), v=v.cuda(), ln=ln, slots=slots))
    side = torch.cuda.Stream()
    for s in sets:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):                # a warm-up on the capture stream
            c.write(s["k"], s["v"], s["slots"])
            c.attention(s["q"], tb, s["ln"])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.write(s["k"], s["v"], s["slots"])
            s["out"] = c.attention(s["q"], tb, s["ln"])
        graphs.append(g)
    torch.cuda.synchronize()
    for s in sets:                                   # other contents, the same addresses
        s["q"].mul_(1.5)
        s["k"].neg_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for s in sets:
        want = c.attention(s["q"], tb, s["ln"])
        assert torch.equal(s["out"], want)
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        got = c.attention(s["q"], tb, s["ln"], stream=other)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    c.check()


def test_decode_loop_of_write_and_attention_together():
    """Forty tokens generated one by one from a converted prompt: each step writes its row and attends to it."""
    rng = np.random.default_rng(13)
    hkv, grp, d, n0, steps = 2, 4, 64, 23, 40
    kp, vp = (to_dtype(rng.normal(size=(6, hkv, 16, d)), torch.bfloat16).cuda() for _ in range(2))
    c = QuantCache(6, hkv, d)
    ids = torch.tensor([4, 0, 5, 2], dtype=torch.int32, device="cuda")
    c.write_pages(kp, vp, ids, ids)
    table = ids[None].contiguous()
    mirror = np.zeros((6, hkv * 18 * d), dtype=np.uint8)
    idh = ids.cpu().numpy()
    slots_all = idh[np.arange(64) // 16] * 16 + np.arange(64) % 16
    rows = [host(x)[idh].transpose(0, 2, 1, 3).reshape(-1, hkv, d) for x in (kp, vp)]
    _kvq.store(mirror, hkv, d, *rows, slots_all)
    for s in range(steps):
        k, v = kv_rows(rng, 1, hkv, d, torch.float32)
        slot = slots_all[n0 + s:n0 + s + 1].astype(np.int32)
        c.write(k.cuda(), v.cuda(), torch.from_numpy(slot).cuda())
        _kvq.store(mirror, hkv, d, host(k), host(v), slot)
        q = to_dtype(rng.normal(size=(1, hkv * grp, d)), torch.float32)
        out = c.attention(q.cuda(), table, torch.tensor([n0 + s + 1], dtype=torch.int32, device="cuda"))
        check_attention(out, mirror, idh[None], q, [n0 + s + 1], hkv)
    assert np.array_equal(c.pool.cpu().numpy(), mirror)
    c.check()


def test_arguments_of_another_kind_are_refused():
    hkv, d = 2, 64
    c = QuantCache(4, hkv, d)
    k = torch.zeros(3, hkv, d, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    for bad in ((k.half(), k.half(), slots), (k, k.float(), slots), (k[:, :1], k[:, :1], slots), (k, k[:2], slots),
                (k.cpu(), k.cpu(), slots), (k, k, slots.long()), (k, k, slots[:2]), (k, k, slots.cpu()),
                (k, k, slots[None])):
        with pytest.raises(ValueError):
            c.write(*bad)
    for bad in ((slots.long(),), (slots, torch.float16), (slots.cpu(),)):
        with pytest.raises(ValueError):
            c.read(*bad)
    pools = torch.zeros(4, hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        c.write_pages(pools, pools, slots, slots[:2])
    with pytest.raises(ValueError):                  # an output is not copied behind the caller's back
        c.read_pages(slots, pools.transpose(2, 3).contiguous().transpose(2, 3), pools, slots)
    q = torch.zeros(1, 4, d, dtype=torch.bfloat16, device="cuda")
    tb, ln = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    for bad in (dict(q=q.half()), dict(q=q[0]), dict(q=q[..., :32]), dict(q=q.cpu()), dict(page_tables=tb.long()),
                dict(page_tables=tb[0]), dict(page_tables=torch.cat([tb, tb])), dict(seq_lens=ln.long()),
                dict(seq_lens=torch.cat([ln, ln])), dict(out=q.float()), dict(out=q[:, :2])):
        with pytest.raises(ValueError):
            c.attention(**{**dict(q=q, page_tables=tb, seq_lens=ln), **bad})
    with pytest.raises(Exception) as e:              # three query heads do not divide over two KV heads
        c.attention(q[:, :3].contiguous(), tb, ln)
    assert "config" in str(e.value)
    c.check()
