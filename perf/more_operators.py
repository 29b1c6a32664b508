"""The paged BF16 cache's operators: the cases they are measured on, their plain
form in elementary torch operations and their exact values in 64 bits.

They work on the key/value pools of one layer, BF16 ``[pages][n_kv_heads][16][d]``
(``persistent_moe_decode_gb300.kv.PagedCache``), and on packed rows: the new
tokens of all sequences one after the other, sequence b's from ``q_starts[b]`` to
``q_starts[b + 1]``.

  rope    rotary positions: of the first r dims of every query and key head,
          pairs (a, b) = (i, i + r / 2), or (2 i, 2 i + 1) interleaved, become
          m (a cos - b sin, a sin + b cos) with the angle position * f_i
  append  the same, the rotated keys and the values going to the cache's slots
          page * 16 + row (a negative slot skips its row), the rotated queries
          in BF16 to the attention
  prompt  causal attention of a sequence's new tokens over all its cached ones,
          the new ones among them: new token i of n sees the first
          seq_len - n + i + 1
  shared  the same where the sequences of a group have their first prefix_len
          tokens in common, on the same pages

Frequencies: f_i = theta^(-2 i / r); linear scaling divides them by a factor; ntk
takes theta factor^(r / (r - 2)) for theta; yarn divides those whose period is
long against the original context (a ramp between beta_slow = 1 and beta_fast = 32
turns in it), keeps the others, and has m = 1 + 0.1 ln(factor).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

PAGE = 16


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the tiny model's heads, a padded batch: part of the head, interleaved, fp32 activations
        dict(name="rope_tiny_part", op="rope", rows=13, hq=4, hkv=2, d=64, dtype="fp32", r=32, interleaved=True,
             theta=1e4, scaling="none", factor=1.0, far=300),
        # one decode step of 16 sequences of up to 32K (30B/3.3B shape)
        dict(name="rope_step_b16", op="rope", rows=16, hq=32, hkv=4, d=128, dtype="bf16", r=128, interleaved=False,
             theta=1e6, scaling="linear", factor=4.0, far=32768),
        # a long prompt with positions scaled for a context of a million
        dict(name="rope_prompt_32k", op="rope", rows=32768, hq=32, hkv=4, d=128, dtype="bf16", r=128,
             interleaved=False, theta=1e6, scaling="yarn", factor=32.0, far=1 << 20),
        # the new rows of a padded step go to their slots
        dict(name="append_step_padded", op="append", rows=13, hq=16, hkv=4, d=128, dtype="fp32", r=128,
             interleaved=False, theta=1e4, scaling="none", factor=1.0, far=8192, skip=5),
        # a prompt's rows rotated and cached as it is admitted
        dict(name="append_prompt_8k", op="append", rows=8191, hq=32, hkv=4, d=128, dtype="bf16", r=128,
             interleaved=False, theta=1e6, scaling="none", factor=1.0, far=8191, skip=0),
        # the tiny model's prompt
        dict(name="prompt_tiny_64", op="prompt", hq=4, hkv=2, d=64, seqs="64/64", spare=0),
        # prompts of different lengths packed (mid model): whole ones, pieces behind a cached part, an idle slot
        dict(name="prompt_packed", op="prompt", hq=16, hkv=4, d=128,
             seqs="64/64,1/1,777/777,0/1000,1501/2048,333/8192,2048/2048,100/116", spare=3),
        # continuous batching: one token each of 15 sequences of 1K to 32K and a 512-token piece of a prompt
        dict(name="prompt_mixed_b16", op="prompt", hq=32, hkv=4, d=128,
             seqs="1/1024,1/32768,1/2999,1/30011,1/5003,1/28001,1/7001,1/26003,512/9001,1/24007,1/11003,1/22003,"
                  "1/13001,1/20011,1/15013,1/17001", spare=2),
        # a whole prompt of 32K (30B/3.3B shape)
        dict(name="prompt_32k", op="prompt", hq=32, hkv=4, d=128, seqs="32768/32768", spare=0),
        # tiny model: two groups, one of them without a common part, an idle slot
        dict(name="shared_tiny", op="shared", hq=4, hkv=2, d=64, groups="64=1/81,1/65,0/70;0=5/9,1/33", spare=1),
        # a decode step of 16 sequences behind one document of 32K
        dict(name="shared_b16", op="shared", hq=32, hkv=4, d=128,
             groups="32768=1/32869,1/33768,1/32784,1/34001,1/33005,1/32999,1/33501,1/34768,1/32800,1/33007,1/32777,"
                    "1/34403,1/33111,1/32769,1/33222,1/33333", spare=2),
        # eight questions of about 200 tokens to one text of 8K (mid model)
        dict(name="shared_questions", op="shared", hq=16, hkv=4, d=128,
             groups="8192=200/8392,131/8323,257/8449,99/8291,311/8503,64/8256,180/8372,222/8414", spare=0),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "prompt", "prompt", "shared", "shared"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    grp = rng.choice([1, 2, 3, 4, 5, 8])
    c = dict(op=op, hq=min(32 // hkv, grp) * hkv, hkv=hkv, d=d)
    if op in ("rope", "append"):
        rows = _spread(rng, 1, 32768)
        c |= dict(rows=rows, dtype=rng.choice(["bf16", "fp32"]) if rows < 16384 else "bf16",
                  r=rng.choice([d, d, d // 2, d // 4]), interleaved=rng.choice([False, True]),
                  theta=rng.choice([1e4, 1e6]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                  factor=rng.choice([2.0, 8.0, 32.0]), far=max(rows, _spread(rng, 64, 1 << 20)))
        if op == "append":
            c["skip"] = rng.choice([0, 0, rows // 3])
        return c
    if op == "prompt":
        seqs = []
        batch = _spread(rng, 1, 16)
        for _ in range(batch):
            new = rng.choice([1, _spread(rng, 1, 16384 // batch)])
            seqs.append([new, new + rng.choice([0, _spread(rng, 1, 16384)])])
        if batch > 2 and rng.random() < 0.5:
            seqs[rng.randrange(batch)][0] = 0
        return c | dict(seqs=",".join(f"{n}/{t}" for n, t in seqs), spare=rng.choice([0, 1, 5]))
    groups = []
    for _ in range(rng.choice([1, 1, 2, 3])):
        prefix = PAGE * _spread(rng, 1, 2048)
        size, most = _spread(rng, 2, 16), rng.choice([1, 1, 128])
        seqs = []
        for _ in range(size):
            new = _spread(rng, 1, most)
            seqs.append(f"{new}/{prefix + new + rng.choice([0, _spread(rng, 1, 2048)])}")
        groups.append(f"{prefix}={','.join(seqs)}")
    return c | dict(groups=";".join(groups), spare=rng.choice([0, 1, 5]))


def _seqs(text):
    return [tuple(int(x) for x in s.split("/")) for s in text.split(",")]


def _groups(case):
    """[(common tokens, [(new tokens, tokens), ...]), ...]; a batch without groups is one sequence each."""
    if case["op"] == "prompt":
        return [(0, [s]) for s in _seqs(case["seqs"])]
    return [(int(g.split("=")[0]), _seqs(g.split("=")[1])) for g in case["groups"].split(";")]


def _dtype(case):
    return torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16


# ------------------------------------------------------------------- inputs

def _rows_state(case, g, st):
    n, hq, hkv, d = case["rows"], case["hq"], case["hkv"], case["d"]
    # one matrix of query, key and value rows, as the projection leaves them; a few large channels among the keys
    x = torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda")
    off = torch.randn(hkv, d, generator=g, device="cuda") * (torch.rand(hkv, d, generator=g, device="cuda") < 0.06) * 4
    x[:, hq:hq + hkv] += off
    st["q"], st["k"], st["v"] = x.to(_dtype(case)).split([hq, hkv, hkv], 1)
    # the last rows of a context of up to `far` tokens; a short call's rows are each of another sequence
    if n <= 16:
        pos = torch.randint(0, case["far"], (n,), generator=g, device="cuda")
    else:
        pos = torch.arange(n, device="cuda") + (case["far"] - n)
    st["positions"] = pos.to(torch.int32)
    if case["op"] == "append":
        pages = -(-n // PAGE) + 3
        shape = (pages, hkv, PAGE, d)
        st["k_pool"] = torch.randn(shape, generator=g, device="cuda").bfloat16()
        st["v_pool"] = torch.randn(shape, generator=g, device="cuda").bfloat16()
        perm = torch.randperm(pages, generator=g, device="cuda")
        tok = torch.arange(n, device="cuda") + int(torch.randint(0, PAGE, (1,), generator=g, device="cuda"))
        slots = perm[tok // PAGE] * PAGE + tok % PAGE
        slots[torch.randperm(n, generator=g, device="cuda")[:case["skip"]]] = -1
        st["slots"] = slots.to(torch.int32)


def _sequences_state(case, g, st):
    hq, hkv, d, groups = case["hq"], case["hkv"], case["d"], _groups(case)
    news = [new for _, seqs in groups for new, _ in seqs]
    lens = [length for _, seqs in groups for _, length in seqs]
    need = sum(prefix // PAGE + sum(-(-(length - prefix) // PAGE) for _, length in seqs) for prefix, seqs in groups)
    pages = need + case["spare"] + 1
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(-(-n // PAGE) for n in lens) + case["spare"]), -1, dtype=torch.int32, device="cuda")
    at = b = 0
    for prefix, seqs in groups:
        common = perm[at:at + prefix // PAGE]
        at += len(common)
        for _, length in seqs:
            mine = perm[at:at + -(-(length - prefix) // PAGE)]
            at += len(mine)
            table[b, :len(common) + len(mine)] = torch.cat([common, mine])
            b += 1
    shape = (pages, hkv, PAGE, d)
    off = torch.randn(hkv, 1, d, generator=g, device="cuda") * (torch.rand(hkv, 1, d, generator=g, device="cuda") < 0.06)
    st["k_pool"] = (torch.randn(shape, generator=g, device="cuda") + 4 * off).bfloat16()
    st["v_pool"] = (torch.randn(shape, generator=g, device="cuda") * 0.5).bfloat16()
    st["q"] = torch.randn(sum(news), hq, d, generator=g, device="cuda").bfloat16()
    st["news"], st["lens"], st["groups"] = news, lens, groups
    st["page_tables"] = table
    st["q_starts"] = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32, device="cuda")
    st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["group_starts"] = torch.tensor([0] + list(np.cumsum([len(s) for _, s in groups])), dtype=torch.int32, device="cuda")
    st["prefix_lens"] = torch.tensor([p for p, _ in groups], dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case=case, op=case["op"])
    rows = case["op"] in ("rope", "append")
    (_rows_state if rows else _sequences_state)(case, g, st)
    if own:
        from persistent_moe_decode_gb300 import kv
        if rows:
            scaling = None if case["scaling"] == "none" else case["scaling"]
            st["rope"] = kv.Rope(case["d"], case["theta"], rotary_dim=case["r"], interleaved=case["interleaved"],
                                 scaling=scaling, factor=case["factor"], original_context=32768)
        if "k_pool" in st:
            st["cache"] = kv.PagedCache.from_pools(st["k_pool"], st["v_pool"])
    return st


# ---------------------------------------------------------------- the passes

def _run_own(st):
    op = st["op"]
    if op == "rope":
        return st["rope"].apply(st["q"], st["k"], st["positions"])
    if op == "append":
        q = st["cache"].append(st["rope"], st["q"], st["k"], st["v"], st["positions"], st["slots"])
        return q, st["k_pool"], st["v_pool"]
    if op == "prompt":
        return st["cache"].attention(st["q"], st["q_starts"], st["page_tables"], st["seq_lens"])
    return st["cache"].shared_attention(st["q"], st["q_starts"], st["page_tables"], st["seq_lens"], st["group_starts"],
                                        st["prefix_lens"])


def _cos_sin(case, positions):
    """cos and sin, times m, [n, 1, r / 2] in fp32 of angles in 64 bits."""
    r, theta, factor = case["r"], case["theta"], case["factor"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    m = 1.0
    if case["scaling"] == "ntk":
        theta = theta * factor ** (r / (r - 2))
    f = theta ** (-2 * i / r)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "yarn":
        # the pair whose angle makes n turns over the original context
        low, high = (r * math.log(32768 / (n * 2 * math.pi)) / (2 * math.log(theta)) for n in (32.0, 1.0))
        low, high = max(0, math.floor(low)), min(r - 1, math.ceil(high))
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        m = 1 + 0.1 * math.log(factor)
    a = positions.double()[:, None, None] * f
    return (a.cos() * m).float(), (a.sin() * m).float()


def _rotate(case, x, cos, sin):
    r = case["r"]
    x = x.float()
    if case["interleaved"]:
        a, b = x[..., :r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _softmax(x):
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _attention(st):
    """One matrix of scores per group for its common tokens, one per sequence for its own."""
    case, q = st["case"], st["q"]
    hkv, d = case["hkv"], case["d"]
    out = torch.empty_like(q)
    q = q.float().unflatten(1, (hkv, -1)) / math.sqrt(d)         # [n, hkv, grp, d]
    tables = st["page_tables"].long()
    at = b = 0
    for prefix, seqs in st["groups"]:
        def cached(seq, lo, hi):
            pages = tables[seq, lo // PAGE:-(-hi // PAGE)]
            return (x[pages].float().transpose(0, 1).flatten(1, 2)[:, None, :hi - lo] for x in (st["k_pool"], st["v_pool"]))

        kp, vp = cached(b, 0, prefix)
        for new, length in seqs:
            k, v = cached(b, prefix, length)
            for lo in range(0, new, 512):                        # a piece of the rows: the scores fit the memory
                hi = min(new, lo + 512)
                seen = length - new + hi - prefix
                rows = q[at + lo:at + hi].permute(1, 2, 0, 3)    # [hkv, grp, rows, d]
                x = torch.matmul(rows, k[:, :, :seen].transpose(-1, -2))
                last = torch.arange(length - new + lo, length - new + hi, device="cuda") - prefix
                x = x.masked_fill(torch.arange(seen, device="cuda") > last[:, None], -math.inf)
                if prefix:
                    x = torch.cat([torch.matmul(rows, kp.transpose(-1, -2)), x], -1)
                p = _softmax(x)
                o = torch.matmul(p[..., prefix:], v[:, :, :seen])
                if prefix:
                    o = o + torch.matmul(p[..., :prefix], vp)
                out[at + lo:at + hi] = o.permute(2, 0, 1, 3).flatten(1, 2).to(out.dtype)
            at += new
            b += 1
    return out


def run(state):
    if own:
        return _run_own(state)
    st, op, case = state, state["op"], state["case"]
    if op in ("prompt", "shared"):
        return _attention(st)
    cos, sin = _cos_sin(case, st["positions"])
    q, k = _rotate(case, st["q"], cos, sin), _rotate(case, st["k"], cos, sin)
    if op == "rope":
        return q.to(st["q"].dtype), k.to(st["k"].dtype)
    live = (st["slots"] >= 0).nonzero().flatten()
    page, row = st["slots"][live].long() // PAGE, st["slots"][live].long() % PAGE
    st["k_pool"][page, :, row] = k[live].bfloat16()
    st["v_pool"][page, :, row] = st["v"][live].bfloat16()
    return q.bfloat16(), st["k_pool"], st["v_pool"]


def _pairs(case):
    """(query, key) pairs of a head, and cached tokens that are seen at all."""
    pairs = tokens = 0
    for prefix, seqs in _groups(case):
        tokens += prefix if any(new for new, _ in seqs) else 0
        for new, length in seqs:
            pairs += new * (length - new) + new * (new + 1) // 2
            tokens += length - prefix if new else 0
    return pairs, tokens


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] in ("rope", "append"):
        n, size = case["rows"], 4 if case["dtype"] == "fp32" else 2
        turned = n * (hq + hkv) * case["r"] * 3
        if case["op"] == "rope":
            return {"bytes": 2 * n * (hq + hkv) * d * size + 4 * n, "flops": turned}
        live = n - case["skip"]
        return {"bytes": (n * hq + 2 * live * hkv) * d * (size + 2) + 8 * n, "flops": turned}
    pairs, tokens = _pairs(case)
    news = sum(new for _, seqs in _groups(case) for new, _ in seqs)
    return {"bytes": 4 * tokens * hkv * d + 4 * news * hq * d + 4 * (-(-tokens // PAGE)), "flops": 4 * pairs * hq * d}


# ----------------------------------------------------------- exact, 64 bits

def _exact_turned(case, x, positions):
    """Each pair as a complex number times m e^(i angle)."""
    r, theta, s = case["r"], case["theta"], case["factor"]
    x, m = x.double().clone(), 1.0
    for i in range(r // 2):
        f = (theta if case["scaling"] != "ntk" else theta * s ** (r / (r - 2))) ** (-2.0 * i / r)
        if case["scaling"] == "linear":
            f /= s
        elif case["scaling"] == "yarn":
            pair = [r / 2 * math.log(32768 / (2 * math.pi * n), theta) for n in (32, 1)]
            lo, hi = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), r - 1)
            share = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f *= share / s + 1 - share
            m = 0.1 * math.log(s) + 1
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
        angle = positions.double() * f
        z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.full_like(angle, m), angle)[:, None]
        x[..., a], x[..., b] = z.real, z.imag
    return x


def _exact_attention(st):
    hkv, d, grp = st["case"]["hkv"], st["case"]["d"], st["case"]["hq"] // st["case"]["hkv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    start = 0
    for b, (new, length) in enumerate(zip(st["news"], st["lens"])):
        t = torch.arange(length, device="cuda")
        page, row = st["page_tables"][b].long()[t // PAGE], t % PAGE
        for h in range(hkv):
            k, v = (st[x][page, h, row].double() for x in ("k_pool", "v_pool"))
            for i in range(0, new, 1024):
                n = min(new - i, 1024)
                seen = length - new + i + n
                mine = st["q"][start + i:start + i + n, h * grp:(h + 1) * grp].double()
                x = torch.einsum("ngd,td->gnt", mine, k[:seen]) * d ** -0.5
                hidden = t[None, :seen] - (length - new + i + torch.arange(n, device="cuda"))[:, None] > 0
                x.masked_fill_(hidden, -math.inf)
                x = x.sub_(torch.logsumexp(x, -1, keepdim=True)).exp_()
                out[start + i:start + i + n, h * grp:(h + 1) * grp] = torch.einsum("gnt,td->ngd", x, v[:seen])
        start += new
    return out


def exact(case, seed):
    if case["op"] in ("prompt", "shared"):
        if work(case)["flops"] > 1.2e13:         # above this the card takes more than about 20 seconds
            return None
        return _exact_attention(prepare(case, seed))
    st = prepare(case, seed)
    q, k = (_exact_turned(case, st[x], st["positions"]) for x in "qk")
    if case["op"] == "rope":
        return q, k
    k_pool, v_pool = st["k_pool"].double(), st["v_pool"].double()
    for i in (st["slots"] >= 0).nonzero().flatten().tolist():
        slot = int(st["slots"][i])
        k_pool[slot // PAGE, :, slot % PAGE] = k[i]
        v_pool[slot // PAGE, :, slot % PAGE] = st["v"][i].double()
    return q, k_pool, v_pool
