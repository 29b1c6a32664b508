"""Drives a synthetic decode workload through the C ABI (no arithmetic here).

``StepRunner`` owns the device weights and KV pools of one workload, the
host-side batch bookkeeping (page tables, lengths, churn) and one decoder
handle; ``step()`` schedules and launches one decode step.
"""
from __future__ import annotations

import numpy as np
import torch

from .configs import Workload
from .kvq import QuantCache, page_bytes
from .mk import Decoder
from .synth import DecodeBatch, kv_layer, make_kv_pools, make_model, refill_pages, refill_rows


def make_kv4_pools(dims, num_pages: int, kv_std: float, seed: int, device) -> torch.Tensor:
    """The 4-bit pools of every layer, [L, pages, page bytes] uint8: those of
    :func:`synth.make_kv_pools`, converted a layer at a time."""
    pools = torch.zeros(dims.n_layers, num_pages, page_bytes(dims.n_kv_heads, dims.head_dim), dtype=torch.uint8,
                        device=device)
    ids = torch.arange(num_pages, dtype=torch.int32, device=device)
    for l in range(dims.n_layers):
        k, v = kv_layer(dims, num_pages, kv_std, seed, l, device)
        QuantCache.from_pool(pools[l], dims.n_kv_heads, dims.head_dim).write_pages(k, v, ids, ids)
    return pools


class StepRunner:
    def __init__(self, wl: Workload, device="cuda", seed: int | None = None, model=None,
                 **cfg_kw):
        self.wl = wl
        self.dims = wl.dims
        self.seed = wl.seed if seed is None else seed
        self.device = torch.device(device)
        self.model = model if model is not None else make_model(wl.dims, self.seed, self.device,
                                                                 wl.expert_format)
        self.batch = DecodeBatch(wl, self.seed)
        if wl.kv_format == "int4":
            self.k_pool, self.v_pool = make_kv4_pools(wl.dims, self.batch.num_pages, wl.kv_std, self.seed,
                                                      self.device), None
        else:
            self.k_pool, self.v_pool = make_kv_pools(wl.dims, self.batch.num_pages, wl.kv_std,
                                                     self.seed, self.device)
        self.dec = Decoder(self.model, self.k_pool, self.v_pool, max_batch=wl.batch,
                           max_pages_per_seq=self.batch.max_pages, **cfg_kw)
        self.logits = torch.empty(wl.batch, wl.dims.vocab, dtype=torch.float32, device=self.device)
        self.step_index = 0

    def schedule(self, stream=None):
        b = self.batch
        b.prepare_step()
        self.dec.schedule(b.tokens, b.page_tables, b.seq_lens, seq_ids=b.seq_ids, stream=stream)

    def launch(self, stream=None):
        self.dec.decode(self.logits, stream)

    def step(self, stream=None):
        self.schedule(stream)
        self.launch(stream)

    def check_status(self):
        rc, err = self.dec.status()
        if rc != 0:
            raise RuntimeError(f"device step failed: {rc} {err.as_dict()}")

    def greedy(self) -> np.ndarray:
        return self.logits.argmax(dim=1).to(torch.int32).cpu().numpy()

    def advance(self, next_tokens, refill: bool = True) -> tuple[int, list[int]] | None:
        """Append the step's token; with churn, retire one sequence and admit one.

        ``refill`` draws fresh K/V for the joining sequence's pages (input
        synthesis).  Without it the pages keep the random K/V they already hold
        (a retired sequence's), which is as good a synthetic prefix and keeps
        the random-number kernels out of a timed loop."""
        self.batch.advance(next_tokens)
        self.step_index += 1
        if self.wl.churn:
            slot, pages = self.batch.churn()
            if refill and self.v_pool is None:
                dst = torch.as_tensor(pages, dtype=torch.int32, device=self.device)
                src = torch.arange(len(pages), dtype=torch.int32, device=self.device)
                for l in range(self.dims.n_layers if pages else 0):
                    k, v = refill_rows(self.dims, len(pages), self.wl.kv_std, self.seed, self.step_index, l,
                                       self.device)
                    QuantCache.from_pool(self.k_pool[l], self.dims.n_kv_heads,
                                         self.dims.head_dim).write_pages(k, v, src, dst)
            elif refill:
                refill_pages(self.k_pool, self.v_pool, pages, self.wl.kv_std, self.seed, self.step_index)
            return slot, pages
        return None

    def close(self):
        self.dec.close()
