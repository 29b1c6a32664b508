"""The 4-bit cache's format and operators restated in numpy, 64 bits: element
by element from the addresses and the rounding rules include/mk.h gives."""
from __future__ import annotations

import numpy as np

PAGE = 16


def bf16_bits(x) -> np.ndarray:
    """BF16 bit patterns (uint16) of values that BF16 holds exactly."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32)
    return (u >> 16).astype(np.uint16)


def bits_value(b) -> np.ndarray:
    with np.errstate(invalid="ignore"):
        return (np.asarray(b).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def _unit(x):
    """Spacing of BF16 numbers around |x| (normal and subnormal)."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126)))
    return np.exp2(e - 7)


def quantise(x):
    """codes [..., d], step, low [..., d / 64] of rows x [..., d] (float64 holding BF16 or fp32 numbers)."""
    g = np.asarray(x, dtype=np.float64).reshape(*np.shape(x)[:-1], -1, 64)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)                        # NaN propagates
        finite = np.isfinite(lo) & np.isfinite(hi)
        lo, hi = np.where(finite, lo, 0.0), np.where(finite, hi, 0.0)
        low = np.floor(lo / _unit(lo)) * _unit(lo)
        over = low < -bits_value(0x7f7f)                     # no BF16 number that low
        span = (hi - low).astype(np.float32)
        bad = ~finite | over | ~np.isfinite(span)
        span = np.where(bad, 0.0, span.astype(np.float64))
        want = span / 15
        step = np.ceil(want / _unit(want)) * _unit(want)
        # the quotient may have rounded across a BF16 number
        step = np.where((step - _unit(step) >= 0) & (15 * (step - _unit(want)) >= span), step - _unit(want), step)
        step = np.where(15 * step < span, step + _unit(want), step)
        step = np.where(span == 0, 0.0, np.maximum(step, 2.0 ** -126))
        diff = (g - low[..., None]).astype(np.float32).astype(np.float64)
        code = np.rint(diff / np.where(step == 0, 1.0, step)[..., None])
        code = np.where((bad | (step == 0))[..., None], 0, np.minimum(code, 15))
        low = np.where(bad, np.nan, low + 0.0)
    return code.astype(np.int64).reshape(np.shape(x)), step, low


def key_at(d, t, i):
    """(byte, odd nibble) of the key code of token t, dim i."""
    ng, g, j = d // 64, i // 64, i % 64
    c, n = j // 16, j % 16
    return t * (d // 2) + 8 * ng * c + 8 * g + n // 2, n % 2


def value_at(d, t, i):
    ng, g, j = d // 64, i // 64, i % 64
    c, u, k = j // 8, j % 8 // 4, j % 4
    return 8 * d + t // 2 * d + 8 * ng * c + 8 * g + 4 * u + 2 * (t % 2) + k // 2, k % 2


def scale_at(d, t, g, value):
    return (17 if value else 16) * d + 4 * (t * (d // 64) + g)


def store(pool, hkv, d, k, v, slots):
    """Write rows k, v [n, hkv, d] into the uint8 pool [pages, page bytes] in place; negative slots are skipped."""
    rec = pool.reshape(pool.shape[0], hkv, 18 * d)
    for x, at, value in ((k, key_at, False), (v, value_at, True)):
        code, step, low = quantise(x)
        for r, s in enumerate(np.asarray(slots)):
            if s < 0:
                continue
            page, t = divmod(int(s), PAGE)
            byte, odd = at(d, t, np.arange(d))
            for o in (0, 1):                                  # the two nibbles of a byte
                e = odd == o
                keep = 0x0f if o else 0xf0
                cur = rec[page][:, byte[e]]
                rec[page][:, byte[e]] = (cur & keep) | (code[r][:, e] << (4 * o)).astype(np.uint8)
            for g in range(d // 64):
                a = scale_at(d, t, g, value)
                low_bits = np.where(np.isnan(low[r, :, g]), 0x7fc0, bf16_bits(low[r, :, g]))
                words = np.stack([bf16_bits(step[r, :, g]), low_bits.astype(np.uint16)], -1)
                rec[page][:, a:a + 4] = np.ascontiguousarray(words).view(np.uint8).reshape(hkv, 4)


def load(pool, hkv, d, slots):
    """(codes, step, low) of keys and of values at slots: [n, hkv, d] int, [n, hkv, d] float64 twice."""
    rec = pool.reshape(pool.shape[0], hkv, 18 * d)
    slots = np.asarray(slots)
    page, t = slots // PAGE, slots % PAGE
    i = np.arange(d)
    out = []
    for at, value in ((key_at, False), (value_at, True)):
        byte, odd = at(d, t[:, None], i[None])
        raw = rec[page[:, None], :, byte].transpose(0, 2, 1)
        code = (raw >> (4 * np.broadcast_to(odd, byte.shape)[:, None]).astype(np.uint8)) & 15
        a = scale_at(d, t[:, None], i[None] // 64, value)
        word = [rec[page[:, None], :, a + j].transpose(0, 2, 1).astype(np.uint32) for j in range(4)]
        step = bits_value(word[0] | (word[1] << 8))
        low = bits_value(word[2] | (word[3] << 8))
        out.append((code.astype(np.int64), step, low))
    return out


def attention(q, keys, values, hkv, scale):
    """Exact attention of q [hq, d] over keys / values (code, step, low) of n tokens, and what bounds its error:
    (out [hq, d], spread [hq, d] = sum p (|step code| + |low|) / sum p, score [hq] = the largest
    sum of absolute terms of a score, in units of log2)."""
    hq, d = q.shape
    n = keys[0].shape[0]
    if n == 0:
        return np.zeros((hq, d)), np.zeros((hq, d)), np.zeros(hq)
    grp = hq // hkv
    out, spread, score = np.zeros((hq, d)), np.zeros((hq, d)), np.zeros(hq)
    for h in range(hq):
        g = h // grp
        kc, ks, kl = (a[:, g] for a in keys)
        vc, vs, vl = (a[:, g] for a in values)
        x = scale * ((ks * kc + kl) @ q[h])
        p = np.exp(x - x.max())
        p /= p.sum()
        out[h] = p @ (vs * vc + vl)
        spread[h] = p @ (vs * vc + np.abs(vl))
        score[h] = scale * np.log2(np.e) * ((ks * kc + np.abs(kl)) @ np.abs(q[h])).max()
    return out, spread, score


def attention_tolerance(out, spread, score, n, d, f32, q_bits=24):
    """How far the kernel may be from ``out``, from its roundings:
    a weight is 2^(x + log2 step): x sums d products in fp32 (at most d + 8 roundings, each at most 2^-23 of the
    sum of absolute terms: the tensor cores may truncate), fp32 queries carry 22 bits; 2^x and log2 are good to
    2^-21; a weight is rounded to 11 bits (BF16 call) or 22 (fp32); the sums over n tokens round once per page
    and once per merge, each at most 2^-22 of the sum of absolute terms; the result is rounded to its type.  Errors
    of numerator and denominator add up: the factor 2.  q_bits = 11: the query was rounded to 11 bits, each of its
    elements by at most 2^-11."""
    weight = np.log(2) * ((d + 8) * 2.0 ** -23 + 2.0 ** -22) * score + 2.0 ** -20
    weight = weight + (2.0 ** -21 if f32 else 2.0 ** -11)
    if q_bits == 11:
        weight = weight + np.log(2) * 2.0 ** -11 * score
    sums = (n / PAGE + 512) * 2.0 ** -22
    half_step = 2.0 ** -24 if f32 else 2.0 ** -8
    return half_step * np.abs(out) + 2 * (weight[:, None] + sums) * spread + 1e-38
