"""GPU checks of the latent calls where inputs are at an edge: tokens that are
not finite, values at the ends of the types' range, layouts of one row or one
head, bounds past their tensors, packs and scratch at their limits."""
import numpy as np
import pytest
import torch

import latent_ref as ref
from sparse_attention_indexer_mxfp4_gb300 import _binding as B
from test_gpu_latent import SCALE, _bf16, _check_prefill, _check_sparse, _clean, _dev, _np, _paged_case, _prefill_case, _sparse_case

pytestmark = pytest.mark.gpu
FMTS = [ref.BF16, ref.FP8]


# ------------------------------------------------------------ e4m3 codes of NaN


@pytest.mark.parametrize("code", [0x7f, 0xff])
@pytest.mark.parametrize("latent,scale", [(3, None), (300, None), (511, 140), (64, 0)])
@pytest.mark.parametrize("H", [16, 32, 64])
def test_nan_code_shows(code, latent, scale, H):
    """A NaN code under any scale is NaN to the read-back and to the attention,
    in its own row only."""
    rng = np.random.default_rng(latent + H)
    page = 64
    pool, slots, indptr, qt, q = _sparse_case(rng, ref.FP8, [70, 90, 80], H, page)
    # the largest finite codes and those of the NaN code's mantissa are ordinary
    for s in slots[::3]:
        pool[s // page, (s % page) * 512:][:512:5] = rng.choice([0x7e, 0xfe, 0x77, 0xf7, 0x6f], 103)
    s = slots[75]
    pool[s // page, (s % page) * 512 + latent] = code
    if scale is not None:
        pool[s // page, page * 640 + (s % page) * 8 + latent // 64] = scale
    out, lse = B.idx_latent_attention(qt, _dev(pool), page, ref.FP8, _dev(slots), _dev(indptr), SCALE)
    _clean()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    _check_sparse(pool, ref.FP8, page, slots, indptr, q, out, lse, rows=[0, 2])
    back = torch.empty(page, 576, dtype=torch.bfloat16, device="cuda")
    B.idx_latent_gather(_dev(pool), page, ref.FP8, _dev(np.array([[s // page]], np.int32)),
                        _dev(np.array([0, page], np.int32)), back)
    _clean()
    assert torch.isnan(back[s % page, latent]) and torch.isnan(back[s % page, :512]).sum() == 1
