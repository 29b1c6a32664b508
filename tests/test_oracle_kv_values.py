"""The oracle over fp32 pools (ORC_KV_F32): with BF16 values it gives the BF16
oracle's step, and it leaves the pools alone."""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

import oracle
from persistent_moe_decode_gb300.configs import TINY
from persistent_moe_decode_gb300.synth import make_kv_pools, make_model
from tests._util import dims_dict, host_pool, host_weights


def test_fp32_pools_of_bf16_values_give_the_bf16_step(oracle_lib):
    d = dataclasses.replace(TINY, vocab=256)
    model = make_model(d, 1)
    kp, vp = make_kv_pools(d, 12, 1.0, 1)
    w = host_weights(model)
    tables = np.array([[3, 7, 1], [0, 11, -1]], dtype=np.int32)
    lens, toks = np.array([37, 15], dtype=np.int32), np.array([5, 200], dtype=np.int32)
    ref = oracle.Oracle(dims_dict(d), w, host_pool(kp), host_pool(vp))
    want = ref.decode_step(toks, lens, tables)
    # the pools after the step, its own new rows among them, as fp32
    f32 = [torch.from_numpy(p.view(np.int16).copy()).view(torch.bfloat16).float().numpy()
           for p in (ref.k_pool, ref.v_pool)]
    got = oracle.Oracle(dims_dict(d), w, *f32)
    keep = got.k_pool.copy(), got.v_pool.copy()
    logits = got.decode_step(toks, lens, tables)
    np.testing.assert_allclose(logits, want, rtol=1e-12, atol=1e-12)
    assert np.array_equal(got.k_pool, keep[0]) and np.array_equal(got.v_pool, keep[1])
    # and the values do matter
    got.v_pool[0, 3, 0, 0] += 1.0
    assert np.abs(got.decode_step(toks, lens, tables) - want).max() > 1e-4
