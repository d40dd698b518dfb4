"""A grouped-head attention layer over the library's calls: the 4-bit paged
cache, the attention of a prompt, the decode steps that follow, over the slots
an indexer step selects or over everything, and the eviction of light tokens.

Keys come rotated (latent.rotate_pairs turns queries and keys alike); the layer
holds what a serving program keeps, the pool of pages."""
from __future__ import annotations

import torch

from . import _binding as B
from .pipeline import IndexerStep

DIM = B.KV4_DIM


class GroupedLayer:
    """heads query heads of 128 elements on kv_heads key heads."""

    def __init__(self, heads, kv_heads, num_pages, page_size, scale=None, device="cuda"):
        if kv_heads <= 0 or heads <= 0 or heads % kv_heads:
            raise ValueError("heads must be a multiple of kv_heads")
        self.heads, self.kv_heads, self.page_size = heads, kv_heads, page_size
        self.scale = DIM ** -0.5 if scale is None else scale
        self.pages = torch.zeros(num_pages, B.kv4_page_bytes(page_size, kv_heads), dtype=torch.uint8,
                                 device=device)

    def _check(self, q):
        if q.dim() != 3 or q.shape[1] != self.heads:
            raise ValueError(f"q must be [rows, {self.heads}, {DIM}]")

    def store(self, k, v, slots, stream=None):
        """New tokens (k, v bf16 [T, kv_heads, 128]) into their slots."""
        if k.dim() != 3 or k.shape[1] != self.kv_heads:
            raise ValueError(f"k must be [tokens, {self.kv_heads}, {DIM}]")
        B.idx_kv4_store(k, v, self.pages, self.page_size, slots, stream=stream)

    def prompt(self, q, k, v, cu, slots, stream=None):
        """Whole prompts, none of it cached before: causal attention of q [T, heads, 128] over
        their own k and v, which go into their slots.  Returns (out, lse)."""
        self._check(q)
        self.store(k, v, slots, stream)
        return B.idx_grouped_prefill(q, k, v, cu, cu, self.scale, stream=stream)

    def chunk(self, q, cu_q, block_table, cu_k, num_tokens, stream=None):
        """Causal attention of later rows of prompts over their sequences' num_tokens = cu_k[-1]
        cached tokens (the rows' own stored before).  Returns (out, lse)."""
        self._check(q)
        with B._on(stream):
            k = torch.empty(num_tokens, self.kv_heads, DIM, dtype=torch.bfloat16, device=q.device)
            v = torch.empty_like(k)
            B.idx_kv4_gather(self.pages, self.page_size, block_table, cu_k, k, v)
            return B.idx_grouped_prefill(q, k, v, cu_q, cu_k, self.scale)

    def decode_slots(self, q, slots, indptr, stream=None):
        """Attention over ragged slots (an indexer step's)."""
        self._check(q)
        return B.idx_kv4_attention(q, self.pages, self.page_size, self.kv_heads, slots, indptr,
                                   self.scale, stream=stream)

    def decode_paged(self, q, block_table, context_lens, next_n, max_model_len, mass=None,
                     stream=None):
        """Attention over whole contexts; with mass (fp32 [B, kv_heads, >= max_model_len]) the
        weights that it gives the tokens are added there."""
        self._check(q)
        with B._on(stream):
            out, lse = B.idx_paged_kv4_attention(q, self.pages, self.page_size, self.kv_heads,
                                                 block_table, context_lens, next_n, self.scale,
                                                 max_model_len)
            if mass is not None:
                B.idx_paged_kv4_weights(q, self.pages, self.page_size, self.kv_heads, block_table,
                                        context_lens, next_n, self.scale, max_model_len, lse, mass)
            return out, lse

    def evict(self, mass, context_lens, budget, recent, block_table, new_table, whole_tokens=False,
              stream=None):
        """Sequences shrunk to `budget` tokens on the pages of new_table (not those they are on).
        An indexer's own keys are not moved with them: decode_paged is the step that follows.
        Returns (keep, new context_lens, new mass)."""
        if mass.dim() != 3 or mass.shape[1] != self.kv_heads:
            raise ValueError(f"mass must be [sequences, {self.kv_heads}, columns]")
        return B.idx_kv4_evict(mass, context_lens, budget, recent, self.pages, self.page_size,
                               block_table, new_table, whole_tokens, stream=stream)


class GroupedDecodeStep:
    """One decode step of a layer: the indexer's logits, top-k and slot map, then the layer's
    attention over exactly those slots.  ``case`` is the indexer's (synth.PagedCase); its block
    table places the layer's cache too, so it is of sequences that were not evicted from."""

    def __init__(self, case, layer: GroupedLayer, q, device="cuda"):
        if case.page_size != layer.page_size or case.num_pages > layer.pages.shape[0]:
            raise ValueError(f"the indexer's {case.num_pages} pages of {case.page_size} tokens are not "
                             f"the layer's {layer.pages.shape[0]} pages of {layer.page_size}")
        layer._check(q)
        self.indexer = IndexerStep(case, device=device)
        self.layer = layer
        self._call = B.prepare_kv4_attention(q, layer.pages, layer.page_size, layer.kv_heads,
                                             self.indexer.slots, self.indexer.indptr, layer.scale)
        self.out, self.lse = self._call.keep[4], self._call.keep[5]

    def run(self, stream=None):
        self.indexer.run(stream)
        self._call(stream)

    @property
    def launches_per_step(self) -> int:
        return self.indexer.launches_per_step + self._call.kernels
