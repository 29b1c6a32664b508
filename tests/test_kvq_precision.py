"""The bound on fp32 calls of the 4-bit cache's attention tells a call that
keeps 22 bits of query and weights from one that keeps 11 (no GPU)."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _kvq, _kvq_fp32


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [5, 16, 100])
@pytest.mark.parametrize("size", [1.0, 8.0])
def test_the_fp32_bound_accepts_22_bits_and_rejects_11(n, d, size):
    rng = np.random.default_rng(n + d)
    pool = np.zeros((-(-n // 16), 18 * d), dtype=np.uint8)
    k, v = (rng.normal(size=(n, 1, d)).astype(np.float32).astype(np.float64) for _ in range(2))
    _kvq.store(pool, 1, d, k, v, np.arange(n))
    keys, values = ([a[:, 0] for a in x] for x in _kvq.load(pool, 1, d, np.arange(n)))
    worst = {}
    for q in _kvq_fp32.queries(rng, 8, 8, d, size):
        out, S, P, E = _kvq_fp32.exact(q, keys, values, d ** -0.5)
        # the same numbers as the other restatement's
        ref = _kvq.attention(q, *([a[:, None] for a in x] for x in (keys, values)), 1, d ** -0.5)[0]
        assert np.allclose(out, ref, rtol=0, atol=1e-12)
        tol = _kvq_fp32.tolerance(out, S, P, E, n)
        assert (tol <= 2.0 ** -14 * P).all()                          # a bound near fp32's own, far below 11 bits
        for bits in ((2, 2), (1, 2), (2, 1), (1, 1)):
            got = _kvq_fp32.emulate(q, keys, values, d ** -0.5, *bits)
            worst.setdefault(bits, []).append((np.abs(got - out) / tol).max(1))
    assert np.max(worst[2, 2]) < 0.5
    # a lost half shows in every head of every sequence
    for bits in ((1, 2), (2, 1), (1, 1)):
        assert np.min(worst[bits]) > 1, bits
