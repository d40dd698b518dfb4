"""The grouped-head calls run together as a serving program runs them: prompts attended to and
stored, later chunks over what was read back, decode rows whose weights are kept, eviction, decode
rows over what stayed; and a decode step over an indexer's own slots."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from sparse_attention_indexer_mxfp4_gb300 import GroupedDecodeStep, GroupedLayer, synth
from sparse_attention_indexer_mxfp4_gb300 import _binding as B

pytestmark = pytest.mark.gpu


def _np(t):
    return t.double().cpu().numpy()


def _place(rng, lens, page, pages):
    need = [-(-n // page) for n in lens]
    perm = rng.permutation(pages).astype(np.int32)
    bt = np.zeros((len(lens), max(need)), np.int32)
    at, slots = 0, []
    for b, n in enumerate(lens):
        bt[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        p = np.arange(n)
        slots.append(bt[b, p // page].astype(np.int64) * page + p % page)
    return bt, slots, perm[at:]


def _prompt(rng, lens, heads, kv_heads):
    t = lambda h: torch.from_numpy(rng.standard_normal((sum(lens), h, 128))).bfloat16().cuda()  # noqa: E731
    return t(heads), t(kv_heads), t(kv_heads)


def test_prompt_decode_evict_decode():
    rng = np.random.default_rng(41)
    lens, heads, kv_heads, page, budget, recent = [700, 130, 64], 12, 3, 64, 96, 16
    layer = GroupedLayer(heads, kv_heads, 30, page)
    bt, slots, spare = _place(rng, lens, page, 30)
    q, k, v = _prompt(rng, lens, heads, kv_heads)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    table, ctx = torch.from_numpy(bt).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = layer.prompt(q, k, v, cu, torch.from_numpy(np.concatenate(slots)).cuda())
    # the same rows over what was read back: keys and values differ by their rounding
    again, _ = layer.chunk(q, cu, table, cu, sum(lens))
    last = (cu[1:] - 1).long()
    mass = torch.zeros(3, kv_heads, max(lens), device="cuda")
    whole, wl = layer.decode_paged(q[last], table, ctx, 1, max(lens), mass=mass)
    flat = torch.from_numpy(np.concatenate([rng.permutation(s) for s in slots]).astype(np.int32)).cuda()
    listed, ll = layer.decode_slots(q[last], flat, cu)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == 0
    pool = layer.pages.cpu().numpy()
    group = heads // kv_heads
    for b, n in enumerate(lens):
        for h in range(kv_heads):
            kk, vv = ref.read(pool, page, kv_heads, slots[b], h)
            hs = slice(h * group, (h + 1) * group)
            want = ref.attend(_np(q[last[b], hs]), kk, vv, layer.scale)
            for o, s in ((whole, wl), (listed, ll)):
                ref.check(_np(o[b, hs]), _np(s[b, hs]), want, n, vmax=10)
            # the read-back's rows, with bf16 weights
            ref.check(_np(again[last[b], hs]), None, want, n, ref.HALF_BF16, 10)
            # and the exact keys and values before
            k0, v0 = _np(k[cu[b]:cu[b + 1], h]), _np(v[cu[b]:cu[b + 1], h])
            ref.check(_np(out[last[b], hs]), _np(lse[last[b], hs]),
                      ref.attend(_np(q[last[b], hs]), k0, v0, layer.scale), n, ref.HALF_BF16, 10)
    # weights sum to one for each head
    assert torch.allclose(mass.sum(2), torch.full((3, kv_heads), float(group), device="cuda"), rtol=1e-4)
    # each head keeps its heaviest tokens, and the rows attend to those
    new = torch.from_numpy(spare[:6].reshape(3, 2).copy()).cuda()
    keep, left, new_mass = layer.evict(mass, ctx, budget, recent, table, new)
    after, al = layer.decode_paged(q[last], new, left, 1, budget, mass=new_mass)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == 0 and left.tolist() == [96, 96, 64]
    kept = keep.cpu().numpy()
    for b in range(3):
        for h in range(kv_heads):
            at = kept[b, h][kept[b, h] >= 0]
            kk, vv = ref.read(pool, page, kv_heads, slots[b][at], h)
            hs = slice(h * group, (h + 1) * group)
            ref.check(_np(after[b, hs]), _np(al[b, hs]), ref.attend(_np(q[last[b], hs]), kk, vv, layer.scale), 96, vmax=10)
            assert mass[b, h, at[:-recent]].min() >= torch.tensor(
                [mass[b, h, t].item() for t in range(lens[b] - recent) if t not in set(at)] or [0.0]).max().item()
    assert torch.allclose(new_mass.sum(2) - group, torch.gather(mass, 2, keep.clamp(min=0).long()).masked_fill(
        keep < 0, 0).sum(2), rtol=1e-4)


def test_decode_step_over_an_indexers_slots():
    rng = np.random.default_rng(42)
    case = synth.paged_case(7, [700, 64, 1500], 2, 64, 128, 64, 2048, pool_factor=1.2, topk=256)
    layer = GroupedLayer(24, 3, case.num_pages, 64)
    pool = ref.make_pool(rng, case.num_pages, 64, 3)
    layer.pages.copy_(torch.from_numpy(pool).cuda())
    q = torch.from_numpy(rng.standard_normal((case.rows, 24, 128))).bfloat16().cuda()
    step = GroupedDecodeStep(case, layer, q)
    step.run()
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == 0 and step.launches_per_step >= 4
    indptr, slots = step.indexer.indptr.cpu().numpy(), step.indexer.slots.cpu().numpy()
    for r in range(case.rows):
        assert indptr[r + 1] - indptr[r] == min(256, case.row_ends()[r])
        for h in range(3):
            k, v = ref.read(pool, 64, 3, slots[indptr[r]:indptr[r + 1]], h)
            hs = slice(8 * h, 8 * h + 8)
            ref.check(_np(step.out[r, hs]), _np(step.lse[r, hs]), ref.attend(_np(q[r, hs]), k, v, layer.scale), 256, vmax=4)
    # the whole step captured and replayed
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.run()
    first = step.out.clone()
    step.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, first)


def test_layer_on_another_stream_and_captured():
    """Every part of a call runs on the stream it is given (the current one is kept busy
    meanwhile), and gives the same when captured and replayed."""
    rng = np.random.default_rng(43)
    lens, page = [700, 70], 64
    layer = GroupedLayer(8, 2, 40, page)
    bt, slots, spare = _place(rng, lens, page, 40)
    q, k, v = _prompt(rng, lens, 8, 2)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    table, ctx = torch.from_numpy(bt).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    at = torch.from_numpy(np.concatenate(slots)).cuda()
    flat, last = at.int(), q[(cu[1:] - 1).long()]
    new = torch.from_numpy(spare[:4].reshape(2, 2).copy()).cuda()
    weight = torch.rand(2, 2, 700, device="cuda")
    calls = [lambda s: layer.prompt(q, k, v, cu, at, stream=s),
             lambda s: layer.chunk(q, cu, table, cu, sum(lens), stream=s),
             lambda s: layer.decode_slots(last, flat, cu, stream=s),
             lambda s: layer.decode_paged(last, table, ctx, 1, max(lens), stream=s),
             lambda s: layer.evict(weight, ctx, 100, 10, table, new, stream=s),
             lambda s: layer.evict(weight, ctx, 100, 10, table, new, whole_tokens=True, stream=s)]
    want = [[x.clone() for x in c(None)] for c in calls]
    side = torch.cuda.Stream()
    for c, w in zip(calls, want):
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)  # a tenth of a second
        got = c(side)
        side.synchronize()
        with torch.cuda.stream(side):
            same = all(torch.equal(x, y) for x, y in zip(got, w))
        torch.cuda.synchronize()
        assert same
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = c(None)
        for x in got:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, w))
    assert B.idx_get_device_status() == 0
