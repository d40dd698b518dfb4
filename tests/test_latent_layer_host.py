"""What LatentLayer and SparseDecodeStep refuse, before anything is made on a device."""
from types import SimpleNamespace

import pytest
import torch

from sparse_attention_indexer_mxfp4_gb300 import LatentLayer, SparseDecodeStep

BF = torch.bfloat16


def _layer(page_size=64, pages=4, uk=(3, 128, 512), uv=(3, 128, 512), dtype=BF):
    return LatentLayer(torch.zeros(uk, dtype=dtype), torch.zeros(uv, dtype=dtype), torch.ones(512), torch.ones(8, 64), pages,
                       page_size)


@pytest.mark.parametrize("wrong", [dict(uk=(3, 96, 512), uv=(3, 160, 512)), dict(uk=(2, 128, 512)), dict(uv=(3, 128, 448)),
                                   dict(uk=(128, 512)), dict(dtype=torch.float32)])
def test_up_projections_of_another_shape(wrong):
    with pytest.raises(ValueError, match="w_uk and w_uv"):
        _layer(**wrong)


def test_layer_holds_its_parts_side_by_side():
    layer = _layer()
    assert layer.heads == 3 and layer.w_up.shape == (512, 3 * 256) and layer.pages.shape[0] == 4


@pytest.mark.parametrize("page_size,pages", [(16, 4), (128, 8), (64, 5)])
def test_step_over_a_cache_of_other_pages(page_size, pages):
    """Slots count in the indexer's pages: a layer of other ones holds other tokens there."""
    case = SimpleNamespace(page_size=page_size, num_pages=pages)
    with pytest.raises(ValueError, match="pages"):
        SparseDecodeStep(case, _layer(), torch.zeros(2, 3, 192, dtype=BF), device="cpu")
