"""The BF16 paged cache's operators restated in 64 bits (torch, any device),
from the definitions in include/mk.h, and what their results may be off by.

Attention: every rounding of the kernel is one of these.  The weights, of at
most 2^-8 relative to themselves (BF16), move a result by 2^-8 A at most, with
A = sum_j softmax_j |v_j|; scores, exponentials and sums are fp32 (a score of
|s| <= 64 is off by less than 2^-13: 128 products, each cut by at most 2^-23 of
the largest |q_i k_i| sum, and 2 exponents' worth of it), less than 2^-11 A
together; the result is rounded to BF16, 2^-8 of itself.

Rotary positions: the place in the turn is cut by 2^-32 and rounded to fp32,
2^-25 of a turn, 1.9e-7 in the angle; sincospi is good to 2 units of 2^-24; a
product and a sum, three roundings of 2^-24, the magnitude's one more: below
2^-20 of |a| + |b| together, and the type's half step of the result.
"""
from __future__ import annotations

import math

import torch

PAGE = 16


def turned(x, positions, r, theta, interleaved, freq=None, magnitude=1.0):
    """Rows x [n, heads, d] rotated, in 64 bits, and the size |a| + |b| of each element's pair."""
    x = x.double()
    out, size = x.clone(), torch.zeros_like(x)
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        f = theta ** (-2.0 * i / r) if freq is None else freq[i]
        t = positions.double() * f
        c, s = (magnitude * t.cos())[:, None], (magnitude * t.sin())[:, None]
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., a] * s + x[..., b] * c
        size[..., a] = size[..., b] = abs(magnitude) * (x[..., a].abs() + x[..., b].abs())
    return out, size


def rope_off(got, want, size):
    """How many times its bound the worst element is off."""
    half = torch.finfo(got.dtype).eps / 2
    bound = half * want.abs() + (1 + half) * 2.0 ** -20 * size + 1e-300
    return float(((got.double() - want).abs() / bound).max()) if got.numel() else 0.0


def gather(pool, table, n, head):
    t = torch.arange(n, device=pool.device)
    return pool[table[t // PAGE].long(), head, t % PAGE].double()


def attention(q, k_pool, v_pool, news, lens, tables, scale=None, prefixes=None, first=None):
    """(result, A) in 64 bits, [n, hq, d]; prefixes[b], first[b]: common tokens, and whose table holds their pages."""
    hkv, d = k_pool.shape[1], q.shape[2]
    grp = q.shape[1] // hkv
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    size = torch.zeros_like(out)
    at = 0
    for b, (new, length) in enumerate(zip(news, lens)):
        table = tables[b].clone()
        if prefixes is not None and prefixes[b]:
            table[:prefixes[b] // PAGE] = tables[first[b], :prefixes[b] // PAGE]
        for h in range(hkv):
            k, v = (gather(p, table, length, h) for p in (k_pool, v_pool))
            for i in range(0, new, 512):
                n = min(512, new - i)
                x = torch.einsum("ngd,td->ngt", q[at + i:at + i + n, h * grp:(h + 1) * grp].double(), k) * scale
                last = length - new + i + torch.arange(n, device=q.device)
                hide = torch.arange(length, device=q.device)[None] > last[:, None]
                w = torch.softmax(x.masked_fill(hide[:, None], -math.inf), -1)
                w = torch.where(hide[:, None], torch.zeros_like(w), w)
                w = torch.where((last < 0)[:, None, None], torch.zeros_like(w), w)
                # a hidden value has no part, whatever it is: 0 times NaN is no 0
                clean = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
                o = torch.einsum("ngt,td->ngd", w, clean)
                for j in (~torch.isfinite(v)).any(1).nonzero().flatten().tolist():
                    o = o + torch.where((last >= j)[:, None, None] & ~torch.isfinite(v[j]), v[j], torch.zeros_like(v[j]))
                out[at + i:at + i + n, h * grp:(h + 1) * grp] = o
                size[at + i:at + i + n, h * grp:(h + 1) * grp] = torch.einsum("ngt,td->ngd", w, clean.abs())
        at += new
    return out, size


def attention_off(got, want, size):
    """How many times its bound the worst element is off; infinite if NaN or infinities differ."""
    g = got.double()
    fine = torch.isfinite(want)
    if not torch.equal(fine, torch.isfinite(g)) or not torch.equal(torch.isnan(want), torch.isnan(g)) \
            or not torch.equal(want[~fine & ~want.isnan()], g[~fine & ~want.isnan()]):
        return math.inf
    bound = 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * (2.0 ** -8 + 2.0 ** -11) * size + 1e-300
    return float(((g - want).abs() / bound)[fine].max()) if fine.any() else 0.0


def batch(news, lens, hkv, d, seed, hq, prefixes=None, groups=None, spare=2, junk=True, device="cuda"):
    """Pools of random rows (NaN and infinities wherever no sequence has a token), shuffled page tables, packed
    queries.  groups: sequence counts of groups whose sequences share their first ``prefixes[g]`` tokens."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    need = [-(-n // PAGE) for n in lens]
    pages = sum(need) + spare + 1
    k = torch.randn(pages, hkv, PAGE, d, generator=g, device=device).bfloat16()
    v = torch.randn(pages, hkv, PAGE, d, generator=g, device=device).bfloat16()
    perm = torch.randperm(pages, generator=g, device=device).int()
    tables = torch.full((len(lens), max(need + [0]) + spare), -7, dtype=torch.int32, device=device)
    held = torch.zeros(pages, PAGE, dtype=torch.bool, device=device)
    at, b = 0, 0
    for gi, count in enumerate(groups or [1] * len(lens)):
        common = (prefixes[gi] if groups else 0) // PAGE
        for j in range(count):
            n = need[b]
            own = 0 if j == 0 else common
            tables[b, own:n] = perm[at:at + n - own]
            at += n - own
            if j:
                tables[b, :common] = 1 << 30          # not read: the first one's are
            t = torch.arange(common * PAGE if j else 0, lens[b], device=device)
            held[tables[b, t // PAGE].long(), t % PAGE] = True
            b += 1
    if junk:
        bad = torch.tensor([math.nan, math.inf, -math.inf], device=device).bfloat16()
        for p in (k, v):
            fill = bad[torch.randint(0, 3, p.shape, generator=g, device=device)]
            p.copy_(torch.where(held[:, None, :, None], p, fill))
    q = torch.randn(sum(news), hq, d, generator=g, device=device).bfloat16()
    starts = torch.tensor([0] + list(torch.tensor(news).cumsum(0)) if news else [0], dtype=torch.int32, device=device)
    return dict(q=q, k=k, v=v, tables=tables, starts=starts,
                lens=torch.tensor(lens, dtype=torch.int32, device=device))
