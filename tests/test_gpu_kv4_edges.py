"""Calls over the 4-bit cache at the ends of what their arguments may be: bounds that descend or
are negative, shares of several tiles, weights that tie or are no numbers, tiny factors."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from sparse_attention_indexer_mxfp4_gb300 import _binding as B
from test_gpu_kv4 import SCALE, _bf16, _check_rows, _clean, _dev, _np, _slots, _table  # noqa: F401

pytestmark = pytest.mark.gpu


def _status():
    torch.cuda.synchronize()
    return B.idx_get_device_status()


@pytest.mark.parametrize("heads,rows", [(1, 6), (2, 6), (5, 6), (8, 2000)])
@pytest.mark.parametrize("last", [-1, -2 ** 31, 0])
def test_gather_bounds_below_zero(heads, rows, last):
    """Nothing is written where the last bound is zero or below it, which is told of."""
    pool = torch.zeros(2, ref.page_stride(16, heads), dtype=torch.uint8, device="cuda")
    bt = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    out = torch.full((rows + 64, heads, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    B.idx_kv4_gather(pool, 16, bt, torch.tensor([0, 3, last], dtype=torch.int32, device="cuda"), out[:rows, :, 0],
                     out[:rows, :, 1])
    assert _status() == (B.DEV_BAD_BOUNDS if last < 0 else 0)
    assert (out == 9).all()
