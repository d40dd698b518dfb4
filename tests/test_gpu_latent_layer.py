"""The latent-attention calls run together as a serving program runs them: a
prompt stored, read back, expanded and attended to; decode rows over the same
cache in the absorbed form; and a decode step over an indexer's own slots."""
import numpy as np
import pytest
import torch

import latent_ref as ref
from sparse_attention_indexer_mxfp4_gb300 import LatentLayer, SparseDecodeStep, synth
from sparse_attention_indexer_mxfp4_gb300 import _binding as B
from sparse_attention_indexer_mxfp4_gb300.latent import rotate_pairs

pytestmark = pytest.mark.gpu


def _layer(rng, heads, pages, page, fmt):
    w = lambda: torch.from_numpy(rng.standard_normal((heads, 128, 512)) / 512 ** 0.5).bfloat16().cuda()  # noqa: E731
    ang = np.arange(4096)[:, None] * 10000.0 ** (-np.arange(32) / 32)
    cs = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    norm = torch.from_numpy((1 + 0.1 * rng.standard_normal(512)).astype(np.float32)).cuda()
    return LatentLayer(w(), w(), norm, cs, pages, page, fmt)


def _prompt(rng, layer, lens, page):
    """Stores prompts of these lengths; returns the block table, kv and positions."""
    need = [-(-n // page) for n in lens]
    perm = rng.permutation(layer.pages.shape[0])[:sum(need)].astype(np.int32)
    bt = np.zeros((len(lens), max(need)), np.int32)
    at, slots, pos = 0, [], []
    for b, n in enumerate(lens):
        bt[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        p = np.arange(n)
        pos.append(p)
        slots.append(bt[b, p // page].astype(np.int64) * page + p % page)
    kv = torch.from_numpy(rng.standard_normal((sum(lens), 576))).bfloat16().cuda()
    pos = torch.from_numpy(np.concatenate(pos).astype(np.int32)).cuda()
    layer.store(kv, pos, torch.from_numpy(np.concatenate(slots)).cuda())
    return torch.from_numpy(bt).cuda(), pos, slots


@pytest.mark.parametrize("fmt", [ref.BF16, ref.FP8])
def test_expanded_and_absorbed_agree(fmt):
    """The expanded rows of a prompt and the absorbed rows of the same queries,
    whole and over listed slots, are one attention computed three ways."""
    rng = np.random.default_rng(31)
    lens, heads, page = [300, 65, 129], 16, 64
    layer = _layer(rng, heads, 20, page, fmt)
    bt, pos, slots = _prompt(rng, layer, lens, page)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    q = torch.from_numpy(rng.standard_normal((sum(lens), heads, 192))).bfloat16().cuda()
    q[..., 128:] = rotate_pairs(q[..., 128:], pos, layer.cos_sin)
    out, lse = layer.prefill(q, cu, bt, cu, sum(lens))
    last = (cu[1:] - 1).long()
    whole, wl = layer.decode_paged(q[last], bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), 1, max(lens))
    flat = torch.from_numpy(np.concatenate([rng.permutation(s) for s in slots]).astype(np.int32)).cuda()
    listed, ll = layer.decode_slots(q[last], flat, cu)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == 0
    # the two absorbed forms differ in the order of their sums alone
    assert torch.allclose(whole.float(), listed.float(), rtol=2 ** -6, atol=2 ** -7)
    assert torch.allclose(wl, ll, rtol=0, atol=1e-4)
    # the expanded form rounds keys and values to bf16, the absorbed one the query's
    # latents and the sums: each by 2^-8 of terms of order one
    assert torch.allclose(out[last].float(), whole.float(), rtol=2 ** -5, atol=2 ** -4)
    assert torch.allclose(lse[last], wl, rtol=0, atol=2 ** -5)


def test_decode_step_over_an_indexers_slots():
    rng = np.random.default_rng(32)
    case = synth.paged_case(7, [700, 64, 1500], 2, 64, 128, 64, 2048, pool_factor=1.2, topk=256)
    layer = _layer(rng, 24, case.num_pages, 64, ref.FP8)
    pool = ref.make_pool(rng, ref.FP8, case.num_pages, 64)
    layer.pages.copy_(torch.from_numpy(pool).cuda())
    q = torch.from_numpy(rng.standard_normal((case.rows, 24, 192))).bfloat16().cuda()
    step = SparseDecodeStep(case, layer, q)
    step.run()
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == 0 and step.launches_per_step >= 4
    indptr, slots = step.indexer.indptr.cpu().numpy(), step.indexer.slots.cpu().numpy()
    qa = step.q.double().cpu().numpy()
    for r in range(case.rows):
        assert indptr[r + 1] - indptr[r] == min(256, case.row_ends()[r])
        tok = ref.read_tokens(pool, ref.FP8, 64, slots[indptr[r]:indptr[r + 1]])
        ref.check(step.out[r].double().cpu().numpy(), step.lse[r].double().cpu().numpy(),
                  ref.attend(qa[r], tok, tok[:, :512], layer.scale))
    # the whole step captured and replayed
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.run()
    first = step.out.clone()
    step.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, first)


def test_layer_on_another_stream():
    """Every part of a call runs on the stream it is given, the library products
    between the kernels among them: the current stream is kept busy meanwhile."""
    rng = np.random.default_rng(33)
    lens, heads, page = [130, 70], 16, 64
    layer = _layer(rng, heads, 8, page, ref.FP8)
    bt, pos, slots = _prompt(rng, layer, lens, page)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    flat = torch.from_numpy(np.concatenate(slots).astype(np.int32)).cuda()
    q = torch.from_numpy(rng.standard_normal((sum(lens), heads, 192))).bfloat16().cuda()
    last = q[(cu[1:] - 1).long()]
    calls = [lambda s: layer.prefill(q, cu, bt, cu, sum(lens), stream=s),
             lambda s: layer.decode_slots(last, flat, cu, stream=s),
             lambda s: layer.decode_paged(last, bt, ctx, 1, max(lens), stream=s)]
    want = [[x.clone() for x in c(None)] for c in calls]
    side = torch.cuda.Stream()
    for c, (out, lse) in zip(calls, want):
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)  # a tenth of a second
        got = c(side)
        side.synchronize()
        with torch.cuda.stream(side):
            same = torch.equal(got[0], out) and torch.equal(got[1], lse)
        torch.cuda.synchronize()
        assert same
