"""Refusals of the latent calls' extension, which need no GPU: what is not a
tensor, wrong types, counts and sizes, for calls and for prepared calls."""
import pytest
import torch

from sparse_attention_indexer_mxfp4_gb300 import _binding as B

BF, I32, I64, U8, F32 = torch.bfloat16, torch.int32, torch.int64, torch.uint8, torch.float32


def _z(*shape, d=I32):
    return torch.zeros(*shape, dtype=d)


def _pool():
    return _z(4, B.latent_page_bytes(64, B.LATENT_FP8), d=U8)


CALLS = {
    "store": (B.idx_latent_store, B.prepare_latent_store,
              lambda: [_z(3, 576, d=BF), _z(3), _z(8, 64, d=F32), _z(512, d=F32), 1e-6, _pool(), 64,
                       _z(3, d=I64), B.LATENT_FP8]),
    "gather": (B.idx_latent_gather, B.prepare_latent_gather,
               lambda: [_pool(), 64, B.LATENT_FP8, _z(2, 3), _z(3), _z(10, 576, d=BF), _z(2)]),
    "attention": (B.idx_latent_attention, B.prepare_latent_attention,
                  lambda: [_z(3, 16, 576, d=BF), _pool(), 64, B.LATENT_FP8, _z(5), _z(4), 0.1]),
    "paged": (B.idx_paged_latent_attention, B.prepare_paged_latent_attention,
              lambda: [_z(4, 16, 576, d=BF), _pool(), 64, B.LATENT_FP8, _z(2, 3), _z(2), 2, 0.1, 192]),
    "prefill": (B.idx_latent_prefill, B.prepare_latent_prefill,
                lambda: [_z(5, 4, 192, d=BF), _z(8, 4, 128, d=BF), _z(8, 64, d=BF), _z(8, 4, 128, d=BF), _z(2), _z(2),
                         0.1]),
}
# (call, argument, what is put in its place)
WRONG = [
    ("store", 0, _z(3, 575, d=BF)), ("store", 0, [1, 2]), ("store", 1, _z(2)), ("store", 1, None),
    ("store", 2, _z(8, 62, d=F32)), ("store", 2, None), ("store", 3, _z(511, d=F32)), ("store", 5, _z(4, 64)),
    ("store", 7, _z(3)), ("store", 7, _z(4, d=I64)), ("store", 6, 1 << 40),
    ("gather", 0, None), ("gather", 3, _z(1, 3)), ("gather", 4, _z(3, d=I64)), ("gather", 4, _z(0)),
    ("gather", 5, _z(10, 576, d=F32)), ("gather", 6, _z(3)),
    ("attention", 0, _z(3, 576, d=BF)), ("attention", 1, _z(4, 8, 8, d=U8)), ("attention", 4, _z(5, d=I64)),
    ("attention", 4, _z(10)[::2]), ("attention", 5, _z(5)),
    ("paged", 4, _z(6)), ("paged", 4, _z(1, 3)), ("paged", 5, _z(4)), ("paged", 6, 3), ("paged", 6, 0),
    ("paged", 8, 1 << 33),
    ("prefill", 0, _z(5, 3, 192, d=BF)), ("prefill", 1, _z(9, 4, 128, d=BF)), ("prefill", 2, _z(8, 32, d=BF)),
    ("prefill", 3, _z(8, 4, 128, d=F32)), ("prefill", 4, _z(3)), ("prefill", 5, _z(2, d=I64)),
]


@pytest.mark.parametrize("name,at,value", WRONG)
def test_wrong_argument(name, at, value):
    call, prepare, good = CALLS[name]
    for f in (call, prepare):
        args = good()
        args[at] = value
        with pytest.raises(ValueError):
            f(*args)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_off_the_gpu(name):
    call, prepare, good = CALLS[name]
    for f in (call, prepare):
        with pytest.raises(ValueError, match="CUDA"):
            f(*good())


@pytest.mark.parametrize("name,out,lse", [("attention", _z(3, 16, 500, d=BF), None), ("attention", None, _z(3, 16)),
                                          ("attention", None, _z(2, 16, d=F32)), ("paged", _z(3, 16, 512, d=BF), None),
                                          ("prefill", _z(5, 4, 128, d=F32), False), ("prefill", None, [1])])
def test_wrong_outputs(name, out, lse):
    call, prepare, good = CALLS[name]
    for f in (call, prepare):
        with pytest.raises(ValueError):
            f(*good(), out=out, lse=lse)


def test_numbers_of_another_kind():
    call, _, good = CALLS["attention"]
    args = good()
    args[6] = "0.1"
    with pytest.raises((TypeError, ValueError)):
        call(*args)
