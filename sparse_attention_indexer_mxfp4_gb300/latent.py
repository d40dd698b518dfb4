"""A latent-attention layer over the library's calls: the paged latent cache,
the expanded attention of a prompt and the absorbed attention of the decode
steps that follow, over the slots an indexer step selects or over everything.

The up-projections are plain library products (torch.matmul); everything else
is a libidx.so call.  The layer holds what a serving program keeps: its
weights, the pool of pages and the scratch."""
from __future__ import annotations

import torch

from . import _binding as B
from .pipeline import IndexerStep

NOPE, ROPE, VDIM, LATENT = 128, B.LATENT_ROPE, 128, B.LATENT_DIM


def rotate_pairs(x, positions, cos_sin):
    """Queries' rotated part: pairs (2i, 2i + 1) of the last ROPE elements of x
    [T, H, ROPE] by the angles of their positions, as idx_latent_store turns the
    keys'."""
    cs = cos_sin[positions.long()][:, None]
    c, s = cs[..., :ROPE // 2], cs[..., ROPE // 2:ROPE]
    a, b = x[..., ::2].float(), x[..., 1::2].float()
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2).to(x.dtype)


class LatentLayer:
    """w_uk [H, 128, 512] and w_uv [H, 128, 512] (bf16) bring a latent to a
    head's key and value; norm_weight fp32 [512]; cos_sin fp32 [P, 64]."""

    def __init__(self, w_uk, w_uv, norm_weight, cos_sin, num_pages, page_size,
                 fmt=B.LATENT_FP8, eps=1e-6, scale=None):
        for w in (w_uk, w_uv):
            if w.dtype != torch.bfloat16 or w.shape != (w_uk.shape[0], NOPE, LATENT):
                raise ValueError(f"w_uk and w_uv must be bfloat16 [H, {NOPE}, {LATENT}]")
        self.w_uk, self.w_uv = w_uk.contiguous(), w_uv.contiguous()
        # one product makes both, side by side for each head: [512, H * 256]
        self.w_up = torch.cat([w_uk, w_uv], 1).reshape(-1, LATENT).t().contiguous()
        self.norm_weight, self.cos_sin, self.eps = norm_weight, cos_sin, eps
        self.heads = w_uk.shape[0]
        self.page_size, self.fmt = page_size, fmt
        self.scale = (NOPE + ROPE) ** -0.5 if scale is None else scale
        self.pages = torch.zeros(num_pages, B.latent_page_bytes(page_size, fmt), dtype=torch.uint8,
                                 device=w_uk.device)

    def store(self, kv, positions, slots, stream=None):
        """New tokens (kv bf16 [T, 576], before norm and rotation) into their slots."""
        B.idx_latent_store(kv, positions, self.cos_sin, self.norm_weight, self.eps, self.pages,
                           self.page_size, slots, self.fmt, stream=stream)

    def prefill(self, q, cu_q, block_table, cu_k, num_tokens, stream=None):
        """Expanded causal attention of prompt rows q bf16 [Tq, H, 192] (the
        last 64 rotated) over their sequences' num_tokens = cu_k[-1] cached
        tokens (fewer set IDX_DEV_BAD_BOUNDS in the device status).  Returns
        (out [Tq, H, 128], lse)."""
        n = num_tokens
        with B._on(stream):  # the products between the calls too
            tokens = torch.empty(n, LATENT + ROPE, dtype=torch.bfloat16, device=q.device)
            B.idx_latent_gather(self.pages, self.page_size, self.fmt, block_table, cu_k, tokens)
            kv = torch.matmul(tokens[:, :LATENT], self.w_up).view(n, self.heads, NOPE + VDIM)
            return B.idx_latent_prefill(q, kv[..., :NOPE], tokens[:, LATENT:], kv[..., NOPE:], cu_q,
                                        cu_k, self.scale)

    def absorb(self, q):
        """q bf16 [R, H, 192] with the key projection taken into it: [R, H, 576]."""
        latent = torch.bmm(q[..., :NOPE].transpose(0, 1), self.w_uk).transpose(0, 1)
        return torch.cat([latent, q[..., NOPE:]], -1)

    def project(self, out):
        """Sums of latents [R, H, 512] to values [R, H, 128]."""
        return torch.bmm(out.transpose(0, 1), self.w_uv.transpose(1, 2)).transpose(0, 1)

    def decode_slots(self, q, slots, indptr, stream=None):
        """Absorbed attention over ragged slots (an indexer step's)."""
        with B._on(stream):
            out, lse = B.idx_latent_attention(self.absorb(q), self.pages, self.page_size, self.fmt,
                                              slots, indptr, self.scale)
            return self.project(out), lse

    def decode_paged(self, q, block_table, context_lens, next_n, max_model_len, stream=None):
        """Absorbed attention over whole contexts."""
        with B._on(stream):
            out, lse = B.idx_paged_latent_attention(self.absorb(q), self.pages, self.page_size,
                                                    self.fmt, block_table, context_lens, next_n,
                                                    self.scale, max_model_len)
            return self.project(out), lse


class SparseDecodeStep:
    """One decode step of a layer: the indexer's logits, top-k and slot map,
    then the layer's attention over exactly those slots.  ``case`` is the
    indexer's (synth.PagedCase); its block table places the latent cache too."""

    def __init__(self, case, layer: LatentLayer, q, device="cuda"):
        if case.page_size != layer.page_size or case.num_pages > layer.pages.shape[0]:
            raise ValueError(f"the indexer's {case.num_pages} pages of {case.page_size} tokens are not "
                             f"the layer's {layer.pages.shape[0]} pages of {layer.page_size}")
        self.indexer = IndexerStep(case, device=device)
        self.layer = layer
        self.q = layer.absorb(q)  # a query's products belong to the layers before
        self._call = B.prepare_latent_attention(
            self.q, layer.pages, layer.page_size, layer.fmt, self.indexer.slots,
            self.indexer.indptr, layer.scale)
        self.out, self.lse = self._call.keep[4], self._call.keep[5]

    def run(self, stream=None):
        self.indexer.run(stream)
        self._call(stream)

    @property
    def launches_per_step(self) -> int:
        return self.indexer.launches_per_step + self._call.kernels
