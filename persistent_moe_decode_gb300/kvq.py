"""The 4-bit KV cache on torch tensors: checks, allocation and streams around
the ``mk_kvq_*`` calls of include/mk.h (no arithmetic here).

A :class:`QuantCache` is the paged pool of one layer, ``[pages][page bytes]``
uint8, in the format include/mk.h documents: groups of 64 dims as
``step * code + low``, 4.5 bits a value.  Rows are written as they are produced
(``write``) or converted from a BF16 pool a page at a time (``write_pages``),
read back (``read``, ``read_pages``) and attended to (``attention``).

Every call runs on ``stream``, by default torch's current stream of the cache's
device, and returns before the kernels have run; it can be captured into a CUDA
graph.  Tensors last used on another stream are the caller's to order, as with
any torch operation.  A call with tensors or a stream of another device, another
type or a wrong shape raises; indexes and lengths are checked on the device
(``check``).
"""
from __future__ import annotations

import torch

from . import mk

PAGE_SIZE = 16
_TYPES = {torch.bfloat16: mk.MK_TYPE_BF16, torch.float32: mk.MK_TYPE_F32}


def page_bytes(n_kv_heads: int, head_dim: int) -> int:
    """Bytes of one 16-token page of all KV heads; raises for a shape that is not supported."""
    n = mk.mk_kvq_page_bytes(n_kv_heads, head_dim)
    if n == 0:
        raise ValueError(f"4-bit cache: {n_kv_heads} KV heads of {head_dim} dims are not supported "
                         "(1 to 1024 heads of 64 or 128 dims)")
    return n


class QuantCache:
    """One layer's 4-bit paged KV cache (``pool``: uint8 ``[pages, page bytes]``, all zeros when new)."""

    def __init__(self, n_pages: int, n_kv_heads: int, head_dim: int, device="cuda"):
        self._attach(torch.zeros(n_pages, page_bytes(n_kv_heads, head_dim), dtype=torch.uint8, device=device),
                     n_kv_heads, head_dim)

    @classmethod
    def from_pool(cls, pool: torch.Tensor, n_kv_heads: int, head_dim: int) -> "QuantCache":
        """A cache over an existing pool (kept referenced, not copied)."""
        self = cls.__new__(cls)
        self._attach(pool, n_kv_heads, head_dim)
        return self

    def _attach(self, pool, n_kv_heads, head_dim):
        if pool.dtype != torch.uint8 or pool.dim() != 2 or not pool.is_contiguous() \
                or pool.shape[1] != page_bytes(n_kv_heads, head_dim) or pool.shape[0] < 1:
            raise ValueError("4-bit cache: the pool is a contiguous uint8 [pages, "
                             f"{page_bytes(n_kv_heads, head_dim)}] tensor, got {pool.dtype} {tuple(pool.shape)}")
        if pool.device.type != "cuda":
            raise ValueError(f"4-bit cache: the pool is on {pool.device}, not on a GPU")
        self.pool, self.n_kv_heads, self.head_dim = pool, n_kv_heads, head_dim
        self._dev, self._ws_bytes = pool.get_device(), {}
        self._inner = {1: (n_kv_heads, head_dim), PAGE_SIZE: (n_kv_heads, PAGE_SIZE, head_dim)}
        self.status = torch.zeros(1, dtype=torch.int32, device=pool.device)
        self._c = mk.mk_kvq_cache(pool=pool.data_ptr(), num_pages=pool.shape[0], n_kv_heads=n_kv_heads,
                                  head_dim=head_dim, status=self.status.data_ptr())

    @property
    def n_pages(self) -> int:
        return self.pool.shape[0]

    def check(self) -> None:
        """Raise MkError if a call so far, on whatever stream, met a page, slot or length out of range (waits for
        the device); clears the record."""
        torch.cuda.synchronize(self._dev)
        code = int(self.status.item())
        if code:
            self.status.zero_()
            torch.cuda.synchronize(self._dev)    # a later call's record, on another stream, comes after
            raise mk.MkError(code, "4-bit cache")

    # ------------------------------------------------------------ arguments

    def _index(self, t, name, n=None):
        if t.dtype is not torch.int32 or t.dim() != 1 or t.get_device() != self._dev \
                or (n is not None and t.shape[0] != n):
            raise ValueError(f"{name}: an int32 vector{f' of {n}' if n is not None else ''} on {self.pool.device}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
        return t if t.is_contiguous() else t.contiguous()

    def _rows(self, k, v, unit, out):
        """mk_kv_rows of k and v, and the tensors it points into."""
        inner, shape, dtype = self._inner[unit], k.shape, k.dtype
        if dtype not in _TYPES or v.dtype is not dtype:
            raise ValueError(f"k, v: BF16 or fp32, both alike, got {dtype} and {v.dtype}")
        if shape[1:] != inner or v.shape != shape or k.get_device() != self._dev or v.get_device() != self._dev:
            raise ValueError(f"k, v: [n, {', '.join(map(str, inner))}] on {self.pool.device}, got {tuple(shape)} on "
                             f"{k.device} and {tuple(v.shape)} on {v.device}")
        s, kp, vp = k.stride(), k.data_ptr(), v.data_ptr()
        odd = 0
        for x in s[:-1]:
            odd |= x
        if s[-1] != 1 or odd & (7 if dtype is torch.bfloat16 else 3) or (kp | vp) & 15 or v.stride() != s:
            if out:
                raise ValueError("k, v: rows of consecutive elements at 16-byte strides, k and v alike")
            k, v = (t.clone(memory_format=torch.contiguous_format) for t in (k, v))
            s, kp, vp = k.stride(), k.data_ptr(), v.data_ptr()
        return mk.mk_kv_rows(kp, vp, _TYPES[dtype], shape[0], s[0], s[0] if unit == 1 else s[2], s[1]), (k, v)

    def _dense(self, t):
        s = t.stride()
        return s[2] == 1 and s[1] == self.head_dim and s[0] % (8 if t.dtype is torch.bfloat16 else 4) == 0 \
            and t.data_ptr() % 16 == 0

    def _run(self, fn, stream, *args):
        """fn(stream pointer, ...) with the cache's device and the call's stream current, for torch's own
        allocations and copies too."""
        if stream is None and torch.cuda.current_device() == self._dev:
            return fn(torch._C._cuda_getCurrentRawStream(self._dev), *args)   # current_stream() costs 2 us more
        if stream is not None and stream.device != self.pool.device:
            raise ValueError(f"stream: one of {self.pool.device}, got one of {stream.device}")
        with torch.cuda.device(self._dev), torch.cuda.stream(stream):    # None: the device's current one
            return fn(torch.cuda.current_stream().cuda_stream, *args)

    # ---------------------------------------------------------------- calls

    def write(self, k, v, slots, stream=None) -> None:
        """Quantise rows k, v ``[n, n_kv_heads, head_dim]`` (BF16 or fp32, any 16-byte strides) into slots
        ``page * 16 + row`` (int32 ``[n]``, distinct; a negative one skips its row)."""
        self._run(self._write, stream, k, v, None, slots, 1)

    def read(self, slots, dtype=torch.bfloat16, stream=None):
        """The keys and values ``[n, n_kv_heads, head_dim]`` at slots ``page * 16 + row``; zeros at a negative one."""
        return self._run(self._read_rows, stream, slots, dtype)

    def write_pages(self, k_pool, v_pool, src_pages, dst_pages, stream=None) -> None:
        """Convert pages ``src_pages`` of BF16 (or fp32) pools ``[pages, n_kv_heads, 16, head_dim]`` into pages
        ``dst_pages`` of the cache (int32 ``[n]``, destinations distinct; a negative index skips its page)."""
        self._run(self._write, stream, k_pool, v_pool, src_pages, dst_pages, PAGE_SIZE)

    def read_pages(self, src_pages, k_pool, v_pool, dst_pages, stream=None) -> None:
        """Read pages ``src_pages`` of the cache back into pages ``dst_pages`` of BF16 (or fp32) pools (int32
        ``[n]``, destinations distinct; a negative source gives zeros, a negative destination skips its page)."""
        self._run(self._read_pages, stream, src_pages, k_pool, v_pool, dst_pages)

    def attention(self, q, page_tables, seq_lens, scale: float | None = None, out=None, stream=None):
        """Attention of one query token per sequence, q ``[batch, n_q_heads, head_dim]`` (BF16 or fp32), over the
        first ``seq_lens[b]`` cached tokens of ``page_tables[b]`` (int32 ``[batch]`` and ``[batch, max_pages]``).
        ``scale`` defaults to head_dim ** -0.5.  A sequence of no tokens gives zeros.  Returns ``out``, a new tensor
        like q unless given; it may be q."""
        return self._run(self._attention, stream, q, page_tables, seq_lens, scale, out)

    def _write(self, st, k, v, src, dst, unit):
        dst = self._index(dst, "slots" if unit == 1 else "dst_pages", k.shape[0] if unit == 1 else None)
        if src is not None:
            src = self._index(src, "src_pages", dst.numel())
        r, keep = self._rows(k, v, unit, False)
        mk.mk_kvq_write(self._c, r, None if src is None else src.data_ptr(), dst.data_ptr(), dst.numel(), unit, st)

    def _read_pages(self, st, src, k, v, dst):
        src = self._index(src, "src_pages")
        dst = self._index(dst, "dst_pages", src.numel())
        r, keep = self._rows(k, v, PAGE_SIZE, True)
        mk.mk_kvq_read(self._c, src.data_ptr(), r, dst.data_ptr(), src.numel(), PAGE_SIZE, st)

    def _read_rows(self, st, slots, dtype):
        if dtype not in _TYPES:
            raise ValueError(f"dtype: BF16 or fp32, got {dtype}")
        slots = self._index(slots, "slots")
        n, (hkv, d) = slots.shape[0], self._inner[1]
        k = torch.empty((n, hkv, d), dtype=dtype, device=slots.device)
        v = torch.empty_like(k)
        r = mk.mk_kv_rows(k.data_ptr(), v.data_ptr(), _TYPES[dtype], n, hkv * d, hkv * d, d)
        mk.mk_kvq_read(self._c, slots.data_ptr(), r, None, n, 1, st)
        return k, v

    def _attention(self, st, q, page_tables, seq_lens, scale, out):
        dev, d, dtype, shape = self._dev, self.head_dim, q.dtype, q.shape
        if len(shape) != 3 or dtype not in _TYPES or q.get_device() != dev or shape[2] != d:
            raise ValueError(f"q: BF16 or fp32 [batch, heads, {d}] on {self.pool.device}, got {dtype} "
                             f"{tuple(shape)} on {q.device}")
        batch, hq, _ = shape
        if page_tables.dtype is not torch.int32 or page_tables.dim() != 2 or page_tables.get_device() != dev \
                or page_tables.shape[0] != batch:
            raise ValueError(f"page_tables: int32 [{batch}, max_pages] on {self.pool.device}, got "
                             f"{page_tables.dtype} {tuple(page_tables.shape)} on {page_tables.device}")
        seq_lens = self._index(seq_lens, "seq_lens", batch)
        if not page_tables.is_contiguous():
            page_tables = page_tables.contiguous()
        if not self._dense(q):
            q = q.clone(memory_format=torch.contiguous_format)
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        elif out.shape != shape or out.dtype is not dtype or out.get_device() != dev or not self._dense(out):
            raise ValueError(f"out: {dtype} {tuple(shape)} on {self.pool.device}, rows of consecutive heads at "
                             "16-byte strides")
        # the workspace belongs to this call's stream, or to the graph that captures it
        max_pages, kind = page_tables.shape[1], _TYPES[dtype]
        n = self._ws_bytes.get((kind, hq, batch, max_pages))     # a function of these alone
        if n is None:
            if len(self._ws_bytes) >= 1024:
                self._ws_bytes.clear()
            n = self._ws_bytes[kind, hq, batch, max_pages] = mk.mk_kvq_workspace(self._c, kind, hq, batch, max_pages)
        ws = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
        mk.mk_kvq_attention(self._c, q.data_ptr(), q.stride(0), out.data_ptr(), out.stride(0), kind, hq, batch,
                            page_tables.data_ptr(), max_pages, seq_lens.data_ptr(), d ** -0.5 if scale is None else scale,
                            ws.data_ptr() if n else None, n, st)
        return out
