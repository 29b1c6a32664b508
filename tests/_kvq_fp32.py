"""What an fp32 call of the 4-bit cache's attention keeps: cases in which the
roundings it may make are few and can be counted, the bound they give, and an
emulation with fewer bits that the bound has to reject.

A query of the cases has one element other than zero in each group of 64 dims,
so a score's products meet no sum but the group's own: what is left are the
splitting of the query and single fp32 roundings."""
from __future__ import annotations

import numpy as np


def queries(rng, batch, heads, d, size):
    """[batch, heads, d] fp32: in every group one element of about ``size`` at a place that runs over the group with
    the head and the sequence, just below half way between two numbers of 11 bits."""
    q = np.zeros((batch, heads, d))
    for b in range(batch):
        for h in range(heads):
            for g in range(d // 64):
                m = rng.integers(0, 64)
                a = size * (1 + (m + 0.49) / 1024) * rng.choice([-1, 1])
                q[b, h, 64 * g + (b * heads + h + 7 * g) % 64] = np.float32(a)
    return q


def _parts(group):
    """step |code - 8| with its sign, and the middle low + 8 step, [n, d]."""
    code, step, low = group
    return step * (code - 8), low + 8 * step


def exact(q, keys, values, scale):
    """(out [heads, d], S, P, E) of one sequence and one KV head: out in 64 bits; S = sum p step |code - 8| and
    P = S + sum p |middle| (p the softmax); E [heads] = how far, relatively, a weight p may be off.

    A weight is 2^u, u = x - r.  x = sum over groups of f (step s) + middle sq with s the one product of a group:
    the query's two halves (2^-22), s from two exact products (1 rounding), the middle (1), step s, the sums (2 each),
    f and sq with scale_log2 (3: the constant, the product, the caller's scale), the last FMA: together at most
    8 roundings of 2^-24 and 2^-22 of T, the sum of the terms' sizes.  u rounds once, |u| <= |x - max| + 8.  ex2 is good
    to 2^-22, and where warps are merged another ex2 with an argument rounded once."""
    ks, km = _parts(keys)
    vs, vm = _parts(values)
    x = scale * np.log2(np.e) * ((ks + km) @ q.T)                     # [n, heads]
    T = scale * np.log2(np.e) * ((np.abs(ks) + np.abs(km)) @ np.abs(q).T).max(0)
    p = np.exp2(x - x.max(0))
    p /= p.sum(0)
    S, P = p.T @ np.abs(vs), p.T @ (np.abs(vs) + np.abs(vm))
    u = (x.max(0) - x.min(0)) + 8
    E = np.log(2) * ((8 * 2.0 ** -24 + 2.0 ** -22) * T + 2 * 2.0 ** -24 * u) + 2 * 2.0 ** -22
    return p.T @ (vs + vm), S, P, E


def tolerance(out, S, P, E, n):
    """How far the call may be from ``out`` for n <= 128 tokens, a page a warp.  Numerator and denominator take the
    weights' error (2 E P).  The products with codes: w = p step rounds once and is split in two halves (2^-22, and
    2^-32 of the largest weight where a half is subnormal); a page's sum on the tensor cores, of at most 16 products
    and the low halves' sum, loses at most 2^-23 of its largest term for each.  p middle: the middle rounds once, the
    sum over a lane's two tokens and eight lanes five times, the sum with the codes' part once; then eight warps and
    at most 16 blocks, one FMA each: 31 roundings of 2^-24, and 29 of the denominator.  Last the division and the type."""
    k = min(n, 16)
    return 2 * E[:, None] * P + (2.0 ** -22 + 2.0 ** -24 + (k + 1) * 2.0 ** -23 + n * 2.0 ** -32) * S \
        + (31 + 29) * 2.0 ** -24 * P + 2 * 2.0 ** -24 * np.abs(out)


def _halves(x, n):
    """x as one or two FP16 numbers."""
    hi = x.astype(np.float16).astype(np.float64)
    return hi if n == 1 else hi + (x - hi).astype(np.float16).astype(np.float64)


def emulate(q, keys, values, scale, q_halves=2, w_halves=2):
    """The call's roundings of query and weights alone, everything else in 64 bits; one half where the call has two is
    what a kernel that dropped or misplaced the low halves would give."""
    ks, km = _parts(keys)
    vs, vm = _parts(values)
    top = np.abs(q).max(1, keepdims=True)
    up = np.exp2(13 - np.floor(np.log2(top)))
    qr = _halves(q * up, q_halves) / up
    x = scale * np.log2(np.e) * (ks @ qr.T + km @ q.T)
    p = np.exp2(x - x.max(0) + 8)
    step = values[1]
    out = np.empty(q.shape)
    for g in range(q.shape[1] // 64):
        c = slice(64 * g, 64 * g + 64)
        w = p * step[:, 64 * g][:, None]
        sc = np.exp2(7 - np.floor(np.log2(w.max(0))))
        wr = _halves(w * sc, w_halves) / sc
        out[:, c] = (wr.T @ (values[0][:, c] - 8) + p.T @ vm[:, c]) / p.sum(0)[:, None]
    return out
