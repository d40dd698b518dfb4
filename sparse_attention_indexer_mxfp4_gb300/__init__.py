"""GB300-native sparse-attention lightning indexer.

The compute path is the C ABI library libidx.so (include/idx.h), built from
hand-written sm_103a CUDA kernels in ``csrc/``; this package only builds it,
loads it and marshals torch tensors into its calls.
"""
from ._binding import (  # noqa: F401
    DEV_BAD_BOUNDS,
    DEV_BAD_PAGE,
    DEV_TIMEOUT,
    FMT_FP8,
    FMT_MXFP4,
    IndexerError,
    LATENT_BF16,
    LATENT_FP8,
    idx_apply_candidate_mask,
    idx_fill_logits_tail,
    idx_get_device_status,
    idx_grouped_prefill,
    idx_kv4_attention,
    idx_kv4_evict,
    idx_kv4_gather,
    idx_kv4_store,
    idx_latent_attention,
    idx_latent_gather,
    idx_latent_prefill,
    idx_latent_store,
    idx_mqa_logits,
    idx_paged_kv4_attention,
    idx_paged_kv4_weights,
    idx_paged_latent_attention,
    idx_paged_mqa_logits,
    idx_row_ends,
    idx_topk,
    idx_topk_ragged_slots,
    idx_topk_to_ragged_slots,
    grouped_prefill_workspace_size,
    kv4_attention_workspace_size,
    kv4_evict_workspace_size,
    kv4_page_bytes,
    latent_attention_workspace_size,
    latent_page_bytes,
    latent_prefill_workspace_size,
    lib,
    library_path,
    version,
)
from .pipeline import IndexerStep, ProducerStep  # noqa: F401
from .latent import LatentLayer, SparseDecodeStep  # noqa: F401
from .grouped import GroupedDecodeStep, GroupedLayer  # noqa: F401
