"""Host checks of the latent calls where a wrong argument would reach the
device: tensors of several devices, scratch that is not one piece, prepared
calls under another device.  The devices are those of tensors without storage."""
import pytest
import torch

from sparse_attention_indexer_mxfp4_gb300 import _binding as B
from test_latent_calls_host import CALLS

BF, U8 = torch.bfloat16, torch.uint8


class Elsewhere(torch.Tensor):
    """A tensor that says it is on a device, without storage."""

    @staticmethod
    def __new__(cls, shape, dtype, device):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise RuntimeError("a tensor without storage was computed with")


def _on(device, t):
    return Elsewhere(t.shape, t.dtype, device)


def _good(name, device="cuda:0"):
    return [_on(device, x) if torch.is_tensor(x) else x for x in CALLS[name][2]()]


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_of_two_devices(name):
    call, prepare, _ = CALLS[name]
    tensors = [i for i, x in enumerate(_good(name)) if torch.is_tensor(x)]
    for f in (call, prepare):
        for i in tensors:
            args = _good(name)
            args[i] = _on("cuda:1", args[i])
            with pytest.raises(ValueError, match="cuda:0 and cuda:1|cuda:1 and cuda:0"):
                f(*args)


@pytest.mark.parametrize("name,out", [("attention", (3, 16, 512)), ("paged", (4, 16, 512)), ("prefill", (5, 4, 128))])
def test_outputs_and_scratch_of_another_device(name, out):
    call, prepare, _ = CALLS[name]
    for f in (call, prepare):
        for more in (dict(out=_on("cuda:1", torch.empty(out, dtype=BF))),
                     dict(lse=_on("cuda:1", torch.empty(out[:2]))),
                     dict(workspace=_on("cuda:1", torch.empty(64, dtype=U8)))):
            with pytest.raises(ValueError, match="cuda:0 and cuda:1"):
                f(*_good(name), **more)


class _Stream:
    def __init__(self, device):
        self.device_index, self.cuda_stream = device, 7


@pytest.mark.parametrize("current,stream,launches", [(0, None, True), (1, None, False), (0, 0, True), (0, 1, False),
                                                     (1, 0, False), (1, 1, False)])
def test_prepared_call_under_another_device(monkeypatch, current, stream, launches):
    made = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(B, "_raw_stream", lambda device: 5)
    p = B.Prepared("idx_latent_store", (1, 2), None, 1, 0)
    p.fn = lambda *a: made.append(a) or 0
    s = None if stream is None else _Stream(stream)
    if launches:
        p(s)
        assert made == [(1, 2, 5 if s is None else 7)]
    else:
        with pytest.raises(ValueError, match="prepared for cuda:0"):
            p(s)
        assert not made


@pytest.mark.parametrize("name", ["attention", "paged", "prefill"])
@pytest.mark.parametrize("ws", [torch.zeros(1, dtype=U8).expand(1 << 24), torch.zeros(1 << 20, dtype=U8)[::2]])
def test_scratch_that_is_not_one_piece(name, ws):
    """Its elements would be counted as bytes that lie one after another."""
    call, prepare, good = CALLS[name]
    for f in (call, prepare):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            f(*good(), workspace=ws)


@pytest.mark.parametrize("name,flag", [("paged", "ctx_per_row"), ("prefill", "causal")])
def test_flag_without_a_truth_value(name, flag):
    """Its own error comes through, and before anything is launched."""
    call, prepare, good = CALLS[name]
    for f in (call, prepare):
        for args in (good(), _good(name)):
            with pytest.raises(RuntimeError, match="Boolean value"):
                f(*args, **{flag: torch.zeros(2)})


def test_scale_past_its_power_of_two():
    """The kernels take the scale times log2(e), which has to be a number."""
    call = {"idx_latent_attention": 15, "idx_paged_latent_attention": 18, "idx_latent_prefill": 20}
    fake = 0x10000
    base = {
        "idx_latent_attention": [fake, 64 * 576, 576, fake, 41472, 10, 64, 1, fake, fake, 1000, 4, 64, 512, 64, 0.1, fake,
                                 64 * 512, 512, fake, 64, None, 0, None],
        "idx_paged_latent_attention": [fake, 64 * 576, 576, fake, 41472, 10, 64, 1, fake, 16, fake, 0, 2, 2, 1000, 64, 512,
                                       64, 0.1, fake, 64 * 512, 512, None, 0, None, 0, None],
        "idx_latent_prefill": [fake, 64 * 192, 192, fake, 64 * 256, 256, fake, 576, fake, 64 * 256, 256, fake, fake, 2, 100,
                               1000, 64, 128, 64, 128, 0.1, 1, fake, 64 * 128, 128, fake, 64, None, 0, None],
    }
    invalid, workspace = 1, 3
    for name, at in call.items():
        for scale, want in ((2.3e38, workspace), (2.4e38, invalid), (3.4e38, invalid)):
            args = list(base[name])
            args[at] = scale
            assert getattr(B.lib(), name)(*args) == want, (name, scale)
