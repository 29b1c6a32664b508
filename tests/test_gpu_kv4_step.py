"""The decode step over a KV cache held in 4 bits (mk_config.kv_format =
MK_KV_INT4): what it writes into the cache, its attention, its logits, the
schedules and the service.

Each step is checked against three things.  The cache after it: the new
token's rows hold its K (RoPE applied) and V within half a step, every other
byte as before.  The attention output of every layer: an exact 64-bit
attention over the cache's own values, from the step's own QKV.  The logits:
the CPU oracle over pools that hold those values (fp32).
"""
from __future__ import annotations

import dataclasses

import numpy as np
import pytest
import torch

import oracle
from persistent_moe_decode_gb300 import mk
from persistent_moe_decode_gb300.configs import TINY, WORKLOADS
from tests import _kvq
from tests._pair import check_logits, oracle_step_following_ties
from tests._util import dims_dict, host_fp8, host_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from persistent_moe_decode_gb300 import build
    build.build()
    oracle.build()


def runner(name, **kw):
    from persistent_moe_decode_gb300.runner import StepRunner
    return StepRunner(WORKLOADS[name], device="cuda", **kw)


def read_back(pools, d):
    """fp32 pools [L, pages, hkv, 16, d] of the cache's values (host arrays), by the cache's own reader."""
    from persistent_moe_decode_gb300.kvq import QuantCache
    L, pages = pools.shape[:2]
    ids = torch.arange(pages, dtype=torch.int32, device="cuda")
    out = [torch.empty(L, pages, d.n_kv_heads, 16, d.head_dim, device="cuda") for _ in range(2)]
    for l in range(L):
        c = QuantCache.from_pool(pools[l], d.n_kv_heads, d.head_dim)
        c.read_pages(ids, out[0][l], out[1][l], ids)
    return [o.cpu().numpy() for o in out]


def rope(x, pos, theta):
    """RoPE (pairs (i, i + d/2)) of rows [..., d], with the fp32 tables the step uses."""
    d = x.shape[-1]
    ang = pos * theta ** (-2.0 * np.arange(d // 2) / d)
    c, s = np.cos(ang).astype(np.float32).astype(np.float64), np.sin(ang).astype(np.float32).astype(np.float64)
    a, b = x[..., :d // 2], x[..., d // 2:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def check_cache_and_attention(run, before, lens, tables, layers):
    d = run.dims
    hq, hkv, dim, B = d.n_q_heads, d.n_kv_heads, d.head_dim, len(lens)
    after = run.k_pool.cpu().numpy()
    for l in range(d.n_layers):
        changed = np.zeros(after[l].shape, dtype=bool).reshape(after.shape[1], hkv, 18 * dim)
        for b, n in enumerate(lens):
            pg, t = int(tables[b, n // 16]), n % 16
            for at in (_kvq.key_at, _kvq.value_at):
                changed[pg][:, at(dim, t, np.arange(dim))[0]] = True
            for v in (False, True):
                for g in range(dim // 64):
                    a = _kvq.scale_at(dim, t, g, v)
                    changed[pg][:, a:a + 4] = True
        same = after[l] == before[l]
        assert same[~changed.reshape(same.shape)].all(), f"layer {l}: bytes outside the new rows changed"
    for l in layers:
        qkv = np.frombuffer(run.dec.scratch(mk.MK_SCRATCH_QKV, l), dtype=np.float32).reshape(B, -1).astype(np.float64)
        att = np.frombuffer(run.dec.scratch(mk.MK_SCRATCH_ATTN, l), dtype=np.float32).reshape(B, hq, dim)
        for b, n in enumerate(lens):
            x = qkv[b].reshape(-1, dim)
            q, k, v = rope(x[:hq], n, d.rope_theta), rope(x[hq:hq + hkv], n, d.rope_theta), x[hq + hkv:]
            i = np.arange(n + 1)
            keys, values = _kvq.load(after[l], hkv, dim, tables[b, i // 16].astype(np.int64) * 16 + i % 16)
            for (code, step, low), want in ((keys, k), (values, v)):
                # half a step; RoPE's own fp32 rounding (two products and a sum) may move a value over a half-way point
                err = np.abs(step[n] * code[n] + low[n] - want)
                assert (err <= 0.5 * step[n] + 2.0 ** -22 * np.abs(want).max() + 1e-30).all(), (l, b, err.max())
                g = want.reshape(hkv, -1, 64)
                span = (g.max(-1) - g.min(-1))[..., None]
                s = step[n].reshape(hkv, -1, 64)
                # the steps are the smallest that cover the group: low and step each round by less than 2^-7
                assert (15 * s <= (span + 2.0 ** -7 * np.abs(g.min(-1))[..., None]) * (1 + 2.0 ** -6) + 1e-30).all()
            ref, spread, score = _kvq.attention(q, keys, values, hkv, dim ** -0.5)
            # weights as in a BF16 call, q rounded to 11 bits, an fp32 result
            tol = _kvq.attention_tolerance(ref, spread, score, n + 1, dim, False, 11) - 2.0 ** -8 * np.abs(ref) \
                + 2.0 ** -23 * np.abs(ref)
            assert (np.abs(att[b] - ref) <= tol).all(), (l, b, float((np.abs(att[b] - ref) / tol).max()))


@pytest.mark.parametrize("name,steps", [("tiny_kv4", 8), ("tiny_b5_kv4", 6), ("tiny_fp8_kv4", 3), ("mid_8k_kv4", 2),
                                        ("mid_b16_kv4", 2)])
def test_step_over_the_4_bit_cache(name, steps):
    run = runner(name)
    d, wl = run.dims, run.wl
    try:
        shape = (d.n_layers, run.k_pool.shape[1], d.n_kv_heads, 16, d.head_dim)
        orc = oracle.Oracle(dims_dict(d), host_weights(run.model), np.zeros(shape, np.float32),
                            np.zeros(shape, np.float32), fp8=host_fp8(run.model))
        agree = pairs = 0
        for s in range(steps):
            before = run.k_pool.cpu().numpy()
            run.schedule()
            tokens, lens, tables = (x.copy() for x in (run.batch.tokens, run.batch.seq_lens, run.batch.page_tables))
            run.launch()
            torch.cuda.synchronize()
            run.check_status()
            layers = range(d.n_layers) if s == 0 and d.n_layers <= 2 else [0, d.n_layers - 1]
            check_cache_and_attention(run, before, lens, tables, layers)
            orc.k_pool[:], orc.v_pool[:] = read_back(run.k_pool, d)
            idx, _ = run.dec.routing()
            gpu = run.logits.double().cpu().numpy()
            ref, _, _ = oracle_step_following_ties(orc, tokens, lens, tables, idx)
            check_logits(gpu, ref, f"{name} step {s}")
            g = gpu.argmax(1).astype(np.int32)
            agree += int((g == ref.argmax(1)).sum())
            pairs += len(g)
            run.advance(g)
        assert agree >= 0.99 * pairs
    finally:
        run.close()


def test_schedules_agree():
    """Every split, role split and wave order: the same cache, logits equal up to the order of the sums."""
    ref = pools = None
    for kw in ({}, dict(kv_split_tokens=64), dict(n_attn_claimers=1), dict(n_attn_claimers=7),
               dict(n_attn_claimers=1 << 20), dict(n_attn_claimers=1 << 20, wave_order=mk.MK_WAVES_INTERLEAVED),
               dict(sm_cap=1), dict(sm_cap=5), dict(trace_records=64)):
        run = runner("tiny_b5_kv4", **kw)
        try:
            run.step()
            torch.cuda.synchronize()
            run.check_status()
            got, pool = run.logits.clone(), run.k_pool.clone()
            if "trace_records" in kw:
                slots = run.dec and mk.mk_read_debug(run.dec.h, mk.MK_DEBUG_NEW_SLOT)
                b = run.batch
                want = [int(b.page_tables[i, n // 16]) * 16 + n % 16 for i, n in enumerate(b.seq_lens)]
                assert slots.tolist() == want
        finally:
            run.close()
        if ref is None:
            ref, pools = got, pool
            continue
        assert torch.equal(pool, pools), kw
        # fp32 sums of the attention's splits in another order, through two layers
        assert (got - ref).abs().max() <= 1e-3 * ref.abs().max(), (kw, float((got - ref).abs().max()))


def test_step_is_repeatable_and_the_static_entry_agrees():
    run = runner("mid_8k_kv4")
    try:
        run.step()
        torch.cuda.synchronize()
        run.check_status()
        ref, pool = run.logits.clone(), run.k_pool.clone()
        for call in (run.dec.decode, run.dec.decode_static, run.dec.decode):
            run.logits.fill_(float("nan"))
            call(run.logits)
            torch.cuda.synchronize()
            run.check_status()
            assert torch.equal(run.logits, ref) and torch.equal(run.k_pool, pool)
    finally:
        run.close()


def test_bad_pages_are_refused_and_the_cache_is_left_alone():
    run = runner("tiny_kv4")
    try:
        b = run.batch
        b.prepare_step()
        before = run.k_pool.clone()
        for bad in (-1, run.k_pool.shape[1]):
            pt = b.page_tables.copy()
            pt[0, 1] = bad
            with pytest.raises(mk.MkError) as e:
                run.dec.schedule(b.tokens, pt, b.seq_lens)
            assert e.value.code == mk.MK_ERR_BAD_PAGE
        torch.cuda.synchronize()
        assert torch.equal(run.k_pool, before)
    finally:
        run.close()


def test_service_over_the_4_bit_cache_gives_the_step_by_step_tokens():
    """Six requests through three slots: the tokens of a step-by-step greedy loop over a copy of the cache."""
    from persistent_moe_decode_gb300.runner import make_kv4_pools
    from persistent_moe_decode_gb300.synth import make_model
    d = dataclasses.replace(TINY)
    n_req, new, slots = 6, 9, 3
    model = make_model(d, 5, torch.device("cuda"))
    per = 8
    pools = make_kv4_pools(d, n_req * per, 1.0, 5, torch.device("cuda"))
    copy = pools.clone()
    rng = np.random.default_rng(3)
    lens = rng.integers(1, per * 16 - new - 1, size=n_req)
    first = rng.integers(0, d.vocab, size=n_req)
    pages = rng.permutation(n_req * per).astype(np.int32).reshape(n_req, per)
    dec = mk.Decoder(model, pools, None, max_batch=slots, max_pages_per_seq=per)
    logits = torch.empty(slots, d.vocab, device="cuda")
    svc = mk.mk_service_create(dec.h, logits.data_ptr())
    try:
        ids = [mk.mk_service_submit(svc, pages[i], int(lens[i]), int(first[i]), new) for i in range(n_req)]
        mk.mk_service_run(svc, 3 * new)
        mk.mk_service_wait(svc)
        got = [mk.mk_service_result(svc, i) for i in ids]
    finally:
        mk.mk_service_destroy(svc)
        dec.close()
    one = mk.Decoder(model, copy, None, max_batch=1, max_pages_per_seq=per)
    try:
        out = torch.empty(1, d.vocab, device="cuda")
        for i in range(n_req):
            tok, toks, near = int(first[i]), [], False
            for s in range(new):
                one.schedule([tok], pages[i:i + 1], [int(lens[i]) + s])
                one.decode(out)
                top = out[0].topk(2)
                near |= bool(top.values[0] - top.values[1] < 1e-3)   # one or several tokens round differently
                tok = int(out[0].argmax())
                toks.append(tok)
            tokens, done = got[i]
            assert done and len(tokens) == new
            assert near or tokens.tolist() == toks, i
    finally:
        one.close()
