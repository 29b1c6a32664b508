"""The BF16 paged KV cache on torch tensors: checks, allocation and streams
around the ``mk_rope_*`` and ``mk_kv_*`` calls of include/mk.h (no arithmetic of
theirs here but the frequencies of the rotary positions).

A :class:`PagedCache` is one layer's pools, BF16 ``[pages, n_kv_heads, 16,
head_dim]`` each, as :class:`persistent_moe_decode_gb300.mk.Decoder` takes them
for all layers: what fills them so that a decode step can go on from there.
``append`` rotates a projection's query and key rows and puts keys and values in
their slots, ``attention`` is the causal attention of packed prompts (or pieces of
prompts, or single tokens) over their sequences' pages, ``shared_attention`` the
same where sequences have a prefix in common.  :class:`Rope` holds the
frequencies, and rotates on its own where the rows go elsewhere (a
:class:`persistent_moe_decode_gb300.kvq.QuantCache`, for instance).

Every call runs on ``stream``, by default torch's current stream of the tensors'
device, and returns before the kernels have run; it can be captured into a CUDA
graph.  Tensors last used on another stream are the caller's to order, as with
any torch operation.  A call with tensors or a stream of another device, another
type or a wrong shape raises; indexes and lengths are checked on the device
(``PagedCache.check``).
"""
from __future__ import annotations

import math

import numpy as np
import torch

from . import mk

PAGE_SIZE = 16
_TYPES = {torch.bfloat16: mk.MK_TYPE_BF16, torch.float32: mk.MK_TYPE_F32}


# the calls' own cost matters beside kernels of a few microseconds: torch's accessors are called once each
_current_device, _raw_stream = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream


def _run(device, index, fn, stream, *args):
    """fn(stream pointer, ...) with the device and the call's stream current, for torch's own allocations and copies
    too."""
    if stream is None and _current_device() == index:
        return fn(_raw_stream(index), *args)                          # current_stream() costs 2 us more
    if stream is not None and stream.device != device:
        raise ValueError(f"stream: one of {device}, got one of {stream.device}")
    with torch.cuda.device(index), torch.cuda.stream(stream):         # None: the device's current one
        return fn(torch.cuda.current_stream().cuda_stream, *args)


def _vector(t, name, device, index, n=None):
    if t.dtype is not torch.int32 or t.dim() != 1 or t.get_device() != index or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name}: an int32 vector{f' of {n}' if n is not None else ''} on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t if t.is_contiguous() else t.contiguous()


def _new(like, dtype=None):
    return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)


def _rows(t, shape, odd):
    """mk_head_rows of a tensor [n, heads, dims] of this shape, or None where its rows do not lie 16-byte aligned
    (``odd``: the strides' bits that may not be set)."""
    s0, s1, s2 = t.stride()
    p = t.data_ptr()
    return None if s2 != 1 or (s0 | s1) & odd or p & 15 else mk.mk_head_rows(p, shape[1], s0, s1)


def frequencies(rotary_dim: int, theta: float, scaling: str | None = None, factor: float = 1.0,
                original_context: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """Angles per position of the ``rotary_dim / 2`` pairs (fp64) and the magnitude of their cos and sin.

    ``theta ** (-2 i / rotary_dim)``, and for contexts ``factor`` times as long as ``original_context``:
    ``"linear"`` divides all by the factor; ``"ntk"`` takes ``theta * factor ** (r / (r - 2))``; ``"yarn"`` divides the
    pairs that make fewer than ``beta_slow`` turns over the original context, keeps those of more than ``beta_fast``,
    goes over from one to the other in between, and has the magnitude ``1 + 0.1 ln(factor)``.
    """
    r, i = rotary_dim, np.arange(rotary_dim // 2, dtype=np.float64)
    if not (math.isfinite(theta) and theta > 1):
        raise ValueError(f"theta: above 1, got {theta}")
    if scaling is None:
        return theta ** (-2 * i / r), 1.0
    if not (math.isfinite(factor) and factor >= 1):
        raise ValueError(f"factor: 1 or more, got {factor}")
    if scaling == "linear":
        return theta ** (-2 * i / r) / factor, 1.0
    if scaling == "ntk":
        return (theta * factor ** (r / (r - 2))) ** (-2 * i / r), 1.0
    if scaling != "yarn":
        raise ValueError(f"scaling: None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    if original_context < 1 or not 0 < beta_slow < beta_fast:
        raise ValueError(f"yarn: an original_context of 1 or more and 0 < beta_slow < beta_fast, got {original_context}, "
                         f"{beta_slow}, {beta_fast}")

    def pair(turns):        # the pair that makes so many turns over the original context
        return r * math.log(original_context / (turns * 2 * math.pi)) / (2 * math.log(theta))

    low, high = max(0, math.floor(pair(beta_fast))), min(r - 1, math.ceil(pair(beta_slow)))
    ramp = np.clip((i - low) / max(high - low, 1e-3), 0, 1)
    f = theta ** (-2 * i / r)
    return f / factor * ramp + f * (1 - ramp), 1 + 0.1 * math.log(factor)


class Rope:
    """Rotary positions of heads of ``head_dim`` (64 or 128) dims, the first ``rotary_dim`` (a multiple of 16; all by
    default) of which turn: pairs ``(i, i + rotary_dim / 2)``, or ``(2 i, 2 i + 1)`` if ``interleaved``.  The other
    arguments are those of :func:`frequencies`.  Angles are exact to fp32 at any int32 position."""

    def __init__(self, head_dim: int, theta: float, rotary_dim: int | None = None, interleaved: bool = False,
                 scaling: str | None = None, factor: float = 1.0, original_context: int = 0, beta_fast: float = 32.0,
                 beta_slow: float = 1.0, device="cuda"):
        r = head_dim if rotary_dim is None else rotary_dim
        if head_dim not in (64, 128) or r < 16 or r > head_dim or r % 16:
            raise ValueError(f"rotary positions: heads of 64 or 128 dims, a multiple of 16 of them turning, got {head_dim} "
                             f"and {r}")
        self.head_dim, self.rotary_dim, self.interleaved = head_dim, r, bool(interleaved)
        freq, self.magnitude = frequencies(r, theta, scaling, factor, original_context, beta_fast, beta_slow)
        # fractions of a turn a position, of 2^64: an angle's place in its turn is then an integer product
        turns = np.array([int(f / (2 * math.pi) * 2.0 ** 64) for f in freq], dtype=np.uint64)
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)
        if self.turns.device.type != "cuda":
            raise ValueError(f"rotary positions: a GPU, got {self.turns.device}")
        self._dev = self.turns.get_device()
        self._c = mk.mk_rope(self.turns.data_ptr(), head_dim, r, int(self.interleaved), self.magnitude)

    def _heads(self, t, name, n, dtype):
        """The tensor, aligned, and its mk_head_rows."""
        shape = t.shape
        if len(shape) != 3 or t.dtype is not dtype or shape[2] != self.head_dim or t.get_device() != self._dev \
                or shape[0] != n or dtype not in _TYPES:
            raise ValueError(f"{name}: BF16 or fp32 rows [{n}, heads, {self.head_dim}] on {self.turns.device}, q, k and v "
                             f"alike, got {t.dtype} {tuple(shape)} on {t.device}")
        odd = 7 if dtype is torch.bfloat16 else 3
        rows = _rows(t, shape, odd)
        if rows is None:
            t = t.clone(memory_format=torch.contiguous_format)
            rows = _rows(t, shape, odd)
        return t, rows

    def _out(self, t, name, like, dtype):
        """mk_head_rows of a given output."""
        rows = None
        if t.shape == like.shape and t.dtype is dtype and t.get_device() == self._dev:
            rows = _rows(t, like.shape, 7 if dtype is torch.bfloat16 else 3)
        if rows is None:
            raise ValueError(f"{name}: {dtype} {tuple(like.shape)} on {self.turns.device}, rows of consecutive elements "
                             f"at 16-byte strides, got {t.dtype} {tuple(t.shape)} on {t.device}")
        return rows

    def apply(self, q, k, positions, out=None, stream=None):
        """Rows q ``[n, heads, head_dim]`` and k ``[n, kv heads, head_dim]`` (BF16 or fp32, alike) turned by
        ``positions`` (int32 ``[n]``): ``(q, k)``, new tensors, or the pair ``out``, which may be the inputs and else
        lies apart from them."""
        return _run(self.turns.device, self._dev, self._apply, stream, q, k, positions, out)

    def _apply(self, st, q, k, positions, out):
        dtype, n, d = q.dtype, q.shape[0], self.head_dim
        given = (q, k)
        q, q_rows = self._heads(q, "q", n, dtype)
        k, k_rows = self._heads(k, "k", n, dtype)
        positions = _vector(positions, "positions", self.turns.device, self._dev, n)
        if out is None:
            qo, ko = _new(q), _new(k)
            hq, hk = q_rows.n_heads, k_rows.n_heads
            q_to, k_to = mk.mk_head_rows(qo.data_ptr(), hq, hq * d, d), mk.mk_head_rows(ko.data_ptr(), hk, hk * d, d)
        else:
            qo, ko = out
            q_to, k_to = self._out(qo, "out[0]", given[0], dtype), self._out(ko, "out[1]", given[1], dtype)
        mk.mk_rope_apply(self._c, n, positions.data_ptr(), _TYPES[dtype], q_rows, k_rows, q_to, k_to, st)
        return qo, ko


class PagedCache:
    """One layer's BF16 paged KV cache: ``k_pool`` and ``v_pool``, ``[pages, n_kv_heads, 16, head_dim]``, zeros when
    new."""

    def __init__(self, n_pages: int, n_kv_heads: int, head_dim: int, device="cuda"):
        shape = (n_pages, n_kv_heads, PAGE_SIZE, head_dim)
        self._attach(torch.zeros(shape, dtype=torch.bfloat16, device=device),
                     torch.zeros(shape, dtype=torch.bfloat16, device=device))

    @classmethod
    def from_pools(cls, k_pool: torch.Tensor, v_pool: torch.Tensor) -> "PagedCache":
        """A cache over existing pools (kept referenced, not copied)."""
        self = cls.__new__(cls)
        self._attach(k_pool, v_pool)
        return self

    def _attach(self, k_pool, v_pool):
        for t, name in ((k_pool, "k_pool"), (v_pool, "v_pool")):
            if t.dtype is not torch.bfloat16 or t.dim() != 4 or not t.is_contiguous() or t.shape != k_pool.shape \
                    or t.shape[0] < 1 or t.shape[0] >= 1 << 26 or not 1 <= t.shape[1] <= 1024 \
                    or t.shape[2] != PAGE_SIZE or t.shape[3] not in (64, 128) or t.data_ptr() & 15:
                raise ValueError(f"{name}: contiguous BF16 [pages, 1 to 1024 KV heads, 16, 64 or 128 dims], both alike, "
                                 f"got {t.dtype} {tuple(t.shape)}")
            if t.device.type != "cuda" or t.device != k_pool.device:
                raise ValueError(f"{name}: both pools on one GPU, got {k_pool.device} and {v_pool.device}")
        self.k_pool, self.v_pool = k_pool, v_pool
        self.n_pages, self.n_kv_heads, _, self.head_dim = k_pool.shape
        self._dev, self._ws_bytes = k_pool.get_device(), {}
        self.status = mk.status_word(k_pool.device)
        self._c = mk.mk_kv_cache(k_pool.data_ptr(), v_pool.data_ptr(), self.n_pages, self.n_kv_heads, self.head_dim,
                                 self.status.data_ptr())

    def check(self) -> None:
        """Raise MkError if a call so far, on whatever stream, met a page, slot, start or length out of range (waits
        for the device); clears the record."""
        torch.cuda.synchronize(self._dev)
        code = int(self.status.item())
        if code:
            self.status.zero_()
            torch.cuda.synchronize(self._dev)    # a later call's record, on another stream, comes after
            raise mk.MkError(code, "paged cache")

    # ---------------------------------------------------------------- calls

    def append(self, rope: Rope, q, k, v, positions, slots, out=None, stream=None):
        """Turn rows q ``[n, heads, head_dim]`` and k ``[n, n_kv_heads, head_dim]`` by ``positions`` (int32 ``[n]``) and
        put the turned keys and the values v (all BF16 or fp32, alike) into slots ``page * 16 + row`` (int32 ``[n]``,
        distinct; a negative one skips its row).  Returns the turned queries in BF16: ``out``, a new tensor unless given,
        which lies apart from the inputs."""
        return _run(self.k_pool.device, self._dev, self._append, stream, rope, q, k, v, positions, slots, out)

    def attention(self, q, q_starts, page_tables, seq_lens, scale: float | None = None, out=None, stream=None):
        """Causal attention of packed rows q (BF16 ``[n, n_q_heads, head_dim]``): rows ``q_starts[b]`` to
        ``q_starts[b + 1]`` (int32 ``[batch + 1]``) are the last tokens of the ``seq_lens[b]`` (int32 ``[batch]``) that
        ``page_tables[b]`` (int32 ``[batch, max_pages]``, up to 2^24 pages) holds, and each sees those up to itself.
        ``scale`` defaults to head_dim ** -0.5.  A row that sees nothing gives zeros, rows of no sequence are left as they
        were (undefined in a new tensor).  Returns ``out``, a new tensor like q unless given; it may be q."""
        return _run(self.k_pool.device, self._dev, self._attention, stream, q, q_starts, page_tables, seq_lens, None, None,
                    scale, out)

    def shared_attention(self, q, q_starts, page_tables, seq_lens, group_starts, prefix_lens,
                         scale: float | None = None, out=None, stream=None):
        """:meth:`attention` where the sequences ``group_starts[g]`` to ``group_starts[g + 1]`` (int32 ``[groups + 1]``,
        from 0 to the batch) share their first ``prefix_lens[g]`` tokens (int32 ``[groups]``; whole pages before each
        one's new tokens, the first of its page table's entries; 0: nothing): these are read once a group.  For the call
        it takes ``8 * (head_dim + 1)`` bytes a row and query head, whatever is shared."""
        return _run(self.k_pool.device, self._dev, self._attention, stream, q, q_starts, page_tables, seq_lens,
                    group_starts, prefix_lens, scale, out)

    def _append(self, st, rope, q, k, v, positions, slots, out):
        dev, device, d = self._dev, self.k_pool.device, self.head_dim
        if rope.head_dim != d or rope._dev != dev:
            raise ValueError(f"rope: one of heads of {d} dims on {device}, got {rope.head_dim} on {rope.turns.device}")
        dtype, n = q.dtype, q.shape[0]
        q, q_rows = rope._heads(q, "q", n, dtype)
        k, k_rows = rope._heads(k, "k", n, dtype)
        v, v_rows = rope._heads(v, "v", n, dtype)
        hkv = self.n_kv_heads
        if k_rows.n_heads != hkv or v_rows.n_heads != hkv:
            raise ValueError(f"k, v: {hkv} KV heads, got {k.shape[1]} and {v.shape[1]}")
        positions = _vector(positions, "positions", device, dev, n)
        slots = _vector(slots, "slots", device, dev, n)
        if out is None:
            out = _new(q, torch.bfloat16)
            hq = q_rows.n_heads
            to = mk.mk_head_rows(out.data_ptr(), hq, hq * d, d)
        else:
            to = rope._out(out, "out", q, torch.bfloat16)
        mk.mk_kv_append(self._c, rope._c, n, positions.data_ptr(), _TYPES[dtype], q_rows, k_rows, v_rows,
                        slots.data_ptr(), to, st)
        return out

    def _dense(self, t, shape):
        """Elements between rows of consecutive heads, 16-byte aligned; 0 if they do not lie so."""
        s0, s1, s2 = t.stride()
        n, heads, d = shape
        if s2 != 1 or (heads > 1 and s1 != d) or s0 & 7 or t.data_ptr() & 15 or (n > 1 and s0 < heads * d):
            return 0
        return s0 if n > 1 else heads * d

    def _attention(self, st, q, q_starts, page_tables, seq_lens, group_starts, prefix_lens, scale, out):
        dev, device, d = self._dev, self.k_pool.device, self.head_dim
        shape = q.shape
        if len(shape) != 3 or q.dtype is not torch.bfloat16 or q.get_device() != dev or shape[2] != d:
            raise ValueError(f"q: BF16 [rows, heads, {d}] on {device}, got {q.dtype} {tuple(shape)} on {q.device}")
        if page_tables.dtype is not torch.int32 or page_tables.dim() != 2 or page_tables.get_device() != dev:
            raise ValueError(f"page_tables: int32 [batch, max_pages] on {device}, got {page_tables.dtype} "
                             f"{tuple(page_tables.shape)} on {page_tables.device}")
        (n, hq, _), (batch, max_pages) = shape, page_tables.shape
        q_starts = _vector(q_starts, "q_starts", device, dev, batch + 1)
        seq_lens = _vector(seq_lens, "seq_lens", device, dev, batch)
        groups, gs, pl = 0, None, None
        if prefix_lens is not None:
            prefix_lens = _vector(prefix_lens, "prefix_lens", device, dev)
            groups = prefix_lens.shape[0]
            group_starts = _vector(group_starts, "group_starts", device, dev, groups + 1)
            if groups == 0 and batch:
                raise ValueError("prefix_lens: the groups hold all sequences, got none")
            gs, pl = group_starts.data_ptr(), prefix_lens.data_ptr()
        if not page_tables.is_contiguous():
            page_tables = page_tables.contiguous()
        q_stride = self._dense(q, shape)
        if not q_stride:
            q = q.clone(memory_format=torch.contiguous_format)
            q_stride = hq * d
        if out is None:
            out, out_stride = _new(q), hq * d
        else:
            out_stride = 0
            if out.shape == shape and out.dtype is torch.bfloat16 and out.get_device() == dev:
                out_stride = self._dense(out, shape)
            if not out_stride and n * hq:
                raise ValueError(f"out: BF16 {tuple(shape)} on {device}, rows of consecutive heads at 16-byte strides")
        # the workspace belongs to this call's stream, or to the graph that captures it
        key = (hq, n, batch, groups)
        ws_bytes = self._ws_bytes.get(key)      # a function of these alone
        if ws_bytes is None:
            if len(self._ws_bytes) >= 1024:
                self._ws_bytes.clear()
            ws_bytes = mk.mk_kv_workspace(self._c, hq, n, batch, groups)
            if ws_bytes:                        # 0: nothing to do, refused, or a device that could not be asked
                self._ws_bytes[key] = ws_bytes
        ws = self.status.new_empty((ws_bytes + 3) // 4) if ws_bytes else None
        mk.mk_kv_attention(self._c, q.data_ptr(), q_stride, out.data_ptr(), out_stride, hq, n, batch, q_starts.data_ptr(),
                           page_tables.data_ptr(), max_pages, seq_lens.data_ptr(), groups, gs, pl,
                           d ** -0.5 if scale is None else scale, ws.data_ptr() if ws_bytes else None, ws_bytes, st)
        return out
