"""GPU parity of the 4-bit cache and the grouped-head calls with plain 64-bit statements
(kv4_ref), at the lengths, head counts, strides and slots where the kernels' tiles end, and with
everything outside the rows poisoned."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
from sparse_attention_indexer_mxfp4_gb300 import _binding as B

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _bf16(x):
    """(device bf16, its values in float64)."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def _np(t):
    return t.double().cpu().numpy()


def _clean():
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == 0


def _table(rng, lens, page, spare=0):
    """Block table [B, blocks] of random pages for these lengths, pages in all, the spare ones."""
    need = [-(-n // page) for n in lens]
    perm = rng.permutation(sum(need) + spare + 1).astype(np.int32)
    bt = np.full((len(lens), max(need + [1])), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt, len(perm), perm[at:at + spare]


def _slots(bt, b, n, page):
    p = np.arange(n)
    return bt[b, p // page].astype(np.int64) * page + p % page


# ------------------------------------------------------------------------ store


@pytest.mark.parametrize("tokens,heads,page,extra", [(1, 1, 64, 0), (5, 3, 1, 16), (67, 8, 48, 32), (300, 2, 64, 0),
                                                     (1001, 5, 16, 0)])
def test_store_and_gather(tokens, heads, page, extra):
    rng = np.random.default_rng(tokens + page)
    bt, pages, _ = _table(rng, [tokens], page)
    x = rng.standard_normal((tokens, 2, heads + 1, 136)) * np.exp(3 * rng.standard_normal((tokens, 2, heads + 1, 1)))
    x[0, 0, 0, :40] = 0  # a group of zeros
    t, v64 = _bf16(x)
    k, v = t[:, 0, :heads, :128], t[:, 1, :heads, :128]
    slots = _slots(bt, 0, tokens, page)
    skip = tokens // 2 if tokens > 1 else -1
    given = slots.copy()
    if skip >= 0:
        given[skip] = -1
    pool0 = rng.integers(0, 256, (pages, ref.page_stride(page, heads, extra)), dtype=np.uint8)
    pool = _dev(pool0)
    B.idx_kv4_store(k, v, pool, page, _dev(given))
    _clean()
    got, want = pool.cpu().numpy(), pool0.copy()
    for i, s in enumerate(given):
        if s < 0:
            continue
        for h in range(heads):
            for side in range(2):
                ref.write(want, page, heads, s, h, side, *ref.quantise(v64[i, side, h, :128]))
    assert np.array_equal(got, want)
    if skip >= 0:  # what it held may be NaN, and comes back as that
        for h in range(heads):
            for side in range(2):
                ref.write(want, page, heads, slots[skip], h, side, np.zeros(128, np.uint8), np.full(4, 127, np.uint8))
        pool = _dev(want)
    # back, in two pieces of one sequence, into wider rows
    cut = tokens // 3
    out = torch.full((tokens + 2, heads, 2, 144), 7.0, dtype=torch.bfloat16, device="cuda")
    a, b = out[:, :, 0, :128], out[:, :, 1, :128]
    B.idx_kv4_gather(pool, page, _dev(np.concatenate([bt, bt])), _dev(np.array([0, cut, tokens], np.int32)), a, b,
                     seq_starts=_dev(np.array([0, cut], np.int32)))
    _clean()
    for h in range(heads):
        kv = ref.read(want, page, heads, slots, h)
        assert np.array_equal(_np(a[:tokens, h]), kv[0]) and np.array_equal(_np(b[:tokens, h]), kv[1])
    assert (out[tokens:] == 7).all() and (out[..., 128:] == 7).all()


def test_store_codes_are_nearest():
    """Around every midpoint, with the group's exponent pinned at 0; and the exponents' borders."""
    mid = (ref.VALUES[1:] + ref.VALUES[:-1]) / 2
    pts = np.concatenate([ref.VALUES, mid, mid * (1 + 2.0 ** -7), mid * (1 - 2.0 ** -8)])
    x = np.zeros((6, 1, 128))
    x[0, 0, :29] = pts
    x[1, 0, :29] = -pts
    x[:2, 0, 31] = 6
    x[2:, 0] = np.array([6.0, 6.0 * (1 + 2.0 ** -7), 3.0, 1e-30])[:, None] * np.linspace(0, 1, 128)
    t, v = _bf16(x)
    pool = torch.zeros(1, ref.page_stride(8, 1), dtype=torch.uint8, device="cuda")
    B.idx_kv4_store(t, -t, pool, 8, torch.arange(6, device="cuda"))
    _clean()
    want = np.zeros(pool.shape, np.uint8)
    for i in range(6):
        ref.write(want, 8, 1, i, 0, 0, *ref.quantise(v[i, 0]))
        ref.write(want, 8, 1, i, 0, 1, *ref.quantise(-v[i, 0]))
    assert np.array_equal(pool.cpu().numpy(), want)


def test_store_what_is_not_finite_and_extremes():
    x = np.ones((3, 1, 128))
    x[0, 0, 5], x[0, 0, 40], x[1, 0, 127] = np.nan, np.inf, -np.inf
    x[2, 0, :32], x[2, 0, 32:64], x[2, 0, 64:] = 3.38e38, 2.0 ** -133, 1.2e-38
    t, v = _bf16(x)
    pool = torch.zeros(1, ref.page_stride(4, 1), dtype=torch.uint8, device="cuda")
    B.idx_kv4_store(t, t, pool, 4, torch.arange(3, device="cuda"))
    _clean()
    k = ref.read(pool.cpu().numpy(), 4, 1, [0, 1, 2], 0)[0]
    assert np.isnan(k[0, :64]).all() and np.isnan(k[1, 96:]).all()
    assert (k[0, 64:] == 1).all() and (k[1, :96] == 1).all()
    want = ref.values(*ref.quantise(v[2, 0]))
    assert np.array_equal(k[2], want)


def test_slots_and_pages_outside_the_pool():
    t = torch.ones(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(2, ref.page_stride(16, 2), dtype=torch.uint8, device="cuda")
    B.idx_kv4_store(t, t, pool, 16, torch.tensor([3, 32, -5, 1 << 40], device="cuda"))
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_PAGE
    back = [torch.full((6, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bt = torch.tensor([[0], [7]], dtype=torch.int32, device="cuda")
    B.idx_kv4_gather(pool, 16, bt, torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda"), *back,
                     seq_starts=torch.tensor([2, 1], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_PAGE
    want = torch.zeros(6, 2, 128)
    want[1], want[5] = 1, 9
    assert torch.equal(back[0].float().cpu(), want) and torch.equal(back[1].float().cpu(), want)
    B.idx_kv4_gather(pool, 16, bt, torch.tensor([0, 3, 9], dtype=torch.int32, device="cuda"), *back)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_PAGE | B.DEV_BAD_BOUNDS


# -------------------------------------------------------------------- attention


def _check_rows(out, lse, q64, pool, page, heads, sets, weight=ref.HALF_F16):
    """sets: for each row its slots (those that count)."""
    group = q64.shape[1] // heads
    for r, slots in enumerate(sets):
        for h in range(heads):
            k, v = ref.read(pool, page, heads, slots, h)
            hs = slice(h * group, (h + 1) * group)
            ref.check(_np(out[r, hs]), None if lse is None else _np(lse[r, hs]),
                      ref.attend(q64[r, hs], k, v, SCALE), len(slots), weight, np.abs(v).max() if v.size else 0)


LISTS = [[1], [0], [31, 32, 33, 0, 127, 128, 129], [513, 0, 1, 700], [2048, 5, 0, 0, 300]]


@pytest.mark.parametrize("lens", LISTS)
@pytest.mark.parametrize("heads,group,page", [(1, 1, 64), (2, 8, 64), (3, 5, 16), (1, 16, 1), (2, 33, 100), (4, 9, 128)])
def test_ragged_slots(lens, heads, group, page):
    rng = np.random.default_rng(sum(lens) + heads * group)
    pages = -(-800 // page) + 1
    pool = ref.make_pool(rng, pages, page, heads, 16, 2)
    sets = [rng.integers(0, 800, n) for n in lens]  # repeated slots among them
    used = np.concatenate(sets) if sum(lens) else np.zeros(0, int)
    ref.poison(pool, page, heads, used)
    q, q64 = _bf16(rng.standard_normal((len(lens), heads * group, 128)) * 2)
    indptr = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    out, lse = B.idx_kv4_attention(q, _dev(pool), page, heads, _dev(used.astype(np.int32)), _dev(indptr), SCALE)
    _clean()
    _check_rows(out, lse, q64, pool, page, heads, sets)


def test_slots_outside_the_pool_are_left_out():
    rng = np.random.default_rng(3)
    pool = ref.make_pool(rng, 4, 16, 2)
    sets = [rng.integers(0, 64, n) for n in (40, 700)]
    bad = [s.copy() for s in sets]
    bad[0][::3], bad[1][5::7] = 64, -1
    bad[1][6::7] = 2 ** 31 - 1
    q, q64 = _bf16(rng.standard_normal((2, 4, 128)))
    out, lse = B.idx_kv4_attention(q, _dev(pool), 16, 2, _dev(np.concatenate(bad).astype(np.int32)),
                                   _dev(np.array([0, 40, 740], np.int32)), SCALE)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_PAGE
    _check_rows(out, lse, q64, pool, 16, 2, [s[(s >= 0) & (s < 64)] for s in bad])


def test_bounds_that_descend():
    """A list of rows with more tokens than its slots is told of and left alone; one that leaves
    the slots is cut."""
    rng = np.random.default_rng(4)
    pool, slots = ref.make_pool(rng, 16, 64, 1), rng.integers(0, 1024, 1000)
    q, q64 = _bf16(rng.standard_normal((20, 2, 128)))
    out = torch.full((20, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    B.idx_kv4_attention(q, _dev(pool), 64, 1, _dev(slots.astype(np.int32)),
                        _dev(np.array([0, 1000] * 10 + [0], np.int32)), SCALE, out=out)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_BOUNDS and (out == 5).all()
    out, lse = B.idx_kv4_attention(q[:2], _dev(pool), 64, 1, _dev(slots.astype(np.int32)),
                                   _dev(np.array([-5, 600, 5000], np.int32)), SCALE)
    _clean()
    _check_rows(out, lse, q64, pool, 64, 1, [slots[:600], slots[600:]])


def _paged_sets(bt, ends, page, next_n):
    return [_slots(bt, r // next_n, e, page) for r, e in enumerate(ends)]


@pytest.mark.parametrize("ctx", [[1], [0, 40, 129], [512, 513, 2, 1000], [3000, 65]])
@pytest.mark.parametrize("next_n,heads,group,page", [(1, 2, 8, 64), (2, 1, 5, 16), (4, 2, 8, 64), (3, 1, 16, 100), (1, 8, 4, 128),
                                                       (2, 3, 3, 32), (1, 2, 12, 96)])
def test_whole_contexts(ctx, next_n, heads, group, page):
    rng = np.random.default_rng(sum(ctx) + next_n)
    bt, pages, _ = _table(rng, ctx, page)
    pool = ref.make_pool(rng, pages, page, heads, 0, 2)
    q, q64 = _bf16(rng.standard_normal((len(ctx) * next_n, heads * group, 128)) * 2)
    ends = [max(0, c - next_n + 1 + j) for c in ctx for j in range(next_n)]
    sets = _paged_sets(bt, ends, page, next_n)
    ref.poison(pool, page, heads, np.concatenate([_slots(bt, b, c, page) for b, c in enumerate(ctx)]))
    out, lse = B.idx_paged_kv4_attention(q, _dev(pool), page, heads, _dev(bt), _dev(np.array(ctx, np.int32)), next_n,
                                         SCALE, bt.shape[1] * page)
    _clean()
    _check_rows(out, lse, q64, pool, page, heads, sets)


def test_lengths_for_each_row_and_a_short_limit():
    rng = np.random.default_rng(8)
    bt, pages, _ = _table(rng, [900, 700], 64)
    pool = ref.make_pool(rng, pages, 64, 2)
    q, q64 = _bf16(rng.standard_normal((4, 8, 128)))
    per = np.array([900, 3, 0, 650], np.int32)
    out, lse = B.idx_paged_kv4_attention(q, _dev(pool), 64, 2, _dev(bt), _dev(per), 2, SCALE, 800, ctx_per_row=True)
    _clean()
    _check_rows(out, lse, q64, pool, 64, 2, _paged_sets(bt, [800, 3, 0, 650], 64, 2))
    out, lse = B.idx_paged_kv4_attention(q, _dev(pool), 64, 2, _dev(bt), _dev(np.array([-4, 1], np.int32)), 2, SCALE, 800)
    _clean()
    _check_rows(out, lse, q64, pool, 64, 2, _paged_sets(bt, [0, 0, 0, 1], 64, 2))


def test_bad_pages_are_left_out():
    rng = np.random.default_rng(9)
    bt, pages, _ = _table(rng, [300], 64)
    pool = ref.make_pool(rng, pages, 64, 1)
    q, q64 = _bf16(rng.standard_normal((1, 8, 128)))
    slots = _slots(bt, 0, 300, 64)
    wrong = bt.copy()
    wrong[0, 1], wrong[0, 3] = -1, pages
    out, lse = B.idx_paged_kv4_attention(q, _dev(pool), 64, 1, _dev(wrong), _dev(np.array([300], np.int32)), 1, SCALE, 320)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_PAGE
    t = np.arange(300) // 64
    _check_rows(out, lse, q64, pool, 64, 1, [slots[(t != 1) & (t != 3)]])


def test_scales_of_any_size():
    """Scales of the values far apart (bf16 weights then), keys and queries of odd sizes."""
    rng = np.random.default_rng(10)
    page, heads, n = 64, 2, 700
    bt, pages, _ = _table(rng, [n], page)
    pool = ref.make_pool(rng, pages, page, heads)
    m = page * heads
    pool[:, m * 132:m * 136] = rng.integers(60, 190, (pages, m * 4)).astype(np.uint8)
    q, q64 = _bf16(rng.standard_normal((1, 16, 128)) * 10.0 ** rng.integers(-6, 3, (1, 16, 1)))
    out, lse = B.idx_paged_kv4_attention(q, _dev(pool), page, heads, _dev(bt), _dev(np.array([n], np.int32)), 1, SCALE, n)
    _clean()
    _check_rows(out, lse, q64, pool, page, heads, [_slots(bt, 0, n, page)], ref.HALF_BF16)


@pytest.mark.parametrize("first", [0, 200])
def test_a_large_value_of_no_weight(first):
    """A token whose values are 2^40 times the others' but which has next to no weight."""
    rng = np.random.default_rng(11)
    page, n = 64, 400
    bt, pages, _ = _table(rng, [n], page)
    pool = ref.make_pool(rng, pages, page, 1, 0, 0)
    q, q64 = _bf16(np.sign(rng.standard_normal((1, 8, 128))) * np.ones((1, 8, 1)))
    q64[:] = q64[:, :1]
    q.copy_(q[:, :1].expand(1, 8, 128).clone())
    slot = _slots(bt, 0, n, page)[first]
    against = np.where(q64[0, 0] > 0, 15, 7).astype(np.uint8)  # -6 times the query's sign
    ref.write(pool, page, 1, slot, 0, 0, against, np.full(4, 125, np.uint8))
    ref.write(pool, page, 1, slot, 0, 1, np.full(128, 7, np.uint8), np.full(4, 165, np.uint8))
    out, lse = B.idx_paged_kv4_attention(q, _dev(pool), page, 1, _dev(bt), _dev(np.array([n], np.int32)), 1, SCALE, n)
    _clean()
    k, v = ref.read(pool, page, 1, _slots(bt, 0, n, page), 0)
    want = ref.attend(q64[0], k, v, SCALE)
    ref.check(_np(out[0]), _np(lse[0]), want, 0, ref.HALF_BF16)
    # its weight is e^(-1.5 * 128 / sqrt(128)) over a sum of some 400 terms: under 2^-32
    assert np.abs(want[0]).max() < 6 * 2.0 ** 38 * 2.0 ** -32


def test_what_is_not_finite():
    """A NaN scale is NaN for the columns that see its token, and no part of the others."""
    rng = np.random.default_rng(12)
    page, heads = 64, 1
    for at, side in [(299, 1), (299, 0), (298, 1), (40, 1), (40, 0)]:
        bt, pages, _ = _table(rng, [300], page)
        pool = ref.make_pool(rng, pages, page, heads)
        slots = _slots(bt, 0, 300, page)
        (b, _) = ref.spans(page, heads, 0, slots[at] % page)[2 + side]
        pool[slots[at] // page, b + 2] = 255
        q, q64 = _bf16(rng.standard_normal((3, 8, 128)))
        out, lse = B.idx_paged_kv4_attention(q, _dev(pool), page, heads, _dev(bt), _dev(np.array([300], np.int32)), 3, SCALE, 300)
        _clean()
        for j, end in enumerate((298, 299, 300)):
            if end <= at:
                k, v = ref.read(pool, page, heads, slots[:end], 0)
                ref.check(_np(out[j]), _np(lse[j]), ref.attend(q64[j], k, v, SCALE), end, ref.HALF_BF16, 100)
            elif side == 0:
                assert torch.isnan(out[j]).all() and torch.isnan(lse[j]).all()
            else:
                assert torch.isnan(out[j][:, 64:96]).all() and torch.isfinite(lse[j]).all()
                assert torch.isfinite(out[j][:, :64]).all() and torch.isfinite(out[j][:, 96:]).all()


def test_growing_scores_and_masks_of_extremes():
    """Scores that rise over the whole list, and queries that are zero or huge."""
    rng = np.random.default_rng(13)
    page, n = 64, 1500
    bt, pages, _ = _table(rng, [n], page)
    pool = ref.make_pool(rng, pages, page, 1)
    slots = _slots(bt, 0, n, page)
    for i, s in enumerate(slots):
        c = np.full(128, 3, np.uint8)
        ref.write(pool, page, 1, s, 0, 0, c, np.full(4, 118 + i // 200, np.uint8))
    q = np.ones((1, 4, 128))
    q[0, 1], q[0, 2] = 0, 40
    q, q64 = _bf16(q)
    out, lse = B.idx_paged_kv4_attention(q, _dev(pool), page, 1, _dev(bt), _dev(np.array([n], np.int32)), 1, SCALE, n)
    _clean()
    _check_rows(out, lse, q64, pool, page, 1, [slots])


def test_strides_outputs_and_scratch():
    rng = np.random.default_rng(14)
    page, heads = 64, 2
    pool = ref.make_pool(rng, 30, page, heads)
    base, q64 = _bf16(rng.standard_normal((10, 3, 200)))
    q = base.transpose(0, 1)[:, :, 40:168]  # heads outermost
    sets = [rng.integers(0, 30 * page, n) for n in (900, 0, 1500)]
    q64 = q64.transpose(1, 0, 2)[:, :, 40:168]
    indptr = _dev(np.array([0, 900, 900, 2400], np.int32))
    slots = _dev(np.concatenate(sets).astype(np.int32))
    box = torch.full((3, 12, 136), 3.0, dtype=torch.bfloat16, device="cuda")
    lbox = torch.full((3, 16), 3.0, device="cuda")
    size = B.kv4_attention_workspace_size(3, 10, heads, 2400)
    ws = torch.full((size + 256,), 77, dtype=torch.uint8, device="cuda")
    out, lse = B.idx_kv4_attention(q, _dev(pool), page, heads, slots, indptr, SCALE, out=box[:, 1:11, :128],
                                   lse=lbox[:, :10], workspace=ws[:size])
    _clean()
    _check_rows(out, lse, q64, pool, page, heads, sets)
    assert (box[:, 0] == 3).all() and (box[:, 11] == 3).all() and (box[..., 128:] == 3).all()
    assert (lbox[:, 10:] == 3).all() and (ws[size:] == 77).all()
    # the same without lse, again and again the same bits
    first = B.idx_kv4_attention(q, _dev(pool), page, heads, slots, indptr, SCALE, lse=False)
    assert first[1] is None
    for _ in range(3):
        again = B.idx_kv4_attention(q, _dev(pool), page, heads, slots, indptr, SCALE)[0]
        assert torch.equal(again, first[0]) and torch.equal(again, out)


def test_few_units_need_no_scratch():
    """A cluster's shared memory holds the sums of few units of few tiles."""
    f = B.kv4_attention_workspace_size
    assert f(1, 16, 2, 20000) == 0 and f(1, 16, 2, 200000) > 0 and f(200, 16, 2, 2048) > 0
    assert f(1, 16, 2, 600) > 0  # too few to pay for a cluster


@pytest.mark.parametrize("n", [129, 640, 2049, 5000, 16384])
@pytest.mark.parametrize("rows,heads,group", [(1, 1, 1), (3, 2, 8), (2, 8, 16), (1, 3, 40), (30, 4, 2)])
def test_units_shared_by_teams(n, rows, heads, group):
    """Every size of a cluster, groups of it with a tile and without, rows without tokens among them."""
    rng = np.random.default_rng(n + rows)
    lens = [n] + [int(x) for x in rng.integers(0, min(n, 600), rows - 1)]
    if rows > 2:
        lens[1] = 0
    page = 64
    pool = ref.make_pool(rng, 40, page, heads, 0, 2)
    sets = [rng.integers(0, 40 * page, m) for m in lens]
    q, q64 = _bf16(rng.standard_normal((rows, heads * group, 128)) * 2)
    indptr = _dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    args = (q, _dev(pool), page, heads, _dev(np.concatenate(sets).astype(np.int32)), indptr, SCALE)
    out, lse = B.idx_kv4_attention(*args)
    _clean()
    some = sorted({0, min(1, rows - 1), rows - 1})
    _check_rows(out[some], lse[some], q64[some], pool, page, heads, [sets[r] for r in some])
    again = B.idx_kv4_attention(*args)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_teams_captured_and_beside_one_another():
    """A cluster's calls captured and replayed, and two of them at once on two streams."""
    rng = np.random.default_rng(50)
    page, heads, n = 64, 2, 9000
    bt, pages, _ = _table(rng, [n, 7000], page)
    pool = _dev(ref.make_pool(rng, pages, page, heads))
    ctx, table = _dev(np.array([n, 7000], np.int32)), _dev(bt)
    qs = [_bf16(rng.standard_normal((2, 16, 128)))[0] for _ in range(2)]
    call = lambda q, s=None: B.idx_paged_kv4_attention(q, pool, page, heads, table, ctx, 1, SCALE, n, stream=s)  # noqa: E731
    assert B.kv4_attention_workspace_size(2, 16, heads, n) == 0
    want = [call(q) for q in qs]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in qs]
    got = [[call(q, s) for q, s in zip(qs, sides)] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for turn in got for g, w in zip(turn, want) for x, y in zip(g, w))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(qs[0])
    for x in out:
        x.zero_()
    graph.replay()
    _clean()
    assert all(torch.equal(x, y) for x, y in zip(out, want[0]))


def test_calls_beside_one_another():
    """Cut rows on two streams, each with scratch of its own, and one scratch for calls in turn."""
    rng = np.random.default_rng(51)
    page, heads = 64, 4
    pool = _dev(ref.make_pool(rng, 60, page, heads))
    slots = _dev(rng.integers(0, 60 * page, 60 * 700).astype(np.int32))
    indptr = _dev((700 * np.arange(61)).astype(np.int32))
    qs = [_bf16(rng.standard_normal((60, 16, 128)))[0] for _ in range(2)]
    size = B.kv4_attention_workspace_size(60, 16, heads, slots.numel())
    assert size > 0
    args = (pool, page, heads, slots, indptr, SCALE)
    want = [B.idx_kv4_attention(q, *args) for q in qs]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in qs]
    got = [[B.idx_kv4_attention(q, *args, stream=s) for q, s in zip(qs, sides)] for _ in range(20)]
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    turns = [B.idx_kv4_attention(q, *args, workspace=ws) for q in qs for _ in range(3)]
    _clean()
    assert all(torch.equal(x, y) for turn in got for g, w in zip(turn, want) for x, y in zip(g, w))
    assert all(torch.equal(x, y) for g, w in zip(turns, [want[0]] * 3 + [want[1]] * 3) for x, y in zip(g, w))


def test_many_sequences():
    """More sequences than a block has threads, most of them empty or short."""
    rng = np.random.default_rng(15)
    lens = rng.integers(0, 40, 300)
    lens[200], lens[7] = 800, 600
    pool = ref.make_pool(rng, 20, 64, 1)
    sets = [rng.integers(0, 1280, n) for n in lens]
    q, q64 = _bf16(rng.standard_normal((300, 2, 128)))
    out, lse = B.idx_kv4_attention(q, _dev(pool), 64, 1, _dev(np.concatenate(sets).astype(np.int32)),
                                   _dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)), SCALE)
    _clean()
    _check_rows(out, lse, q64, pool, 64, 1, sets)


def test_pages_past_32_bits():
    """Pages at byte offsets over 2^32."""
    rng = np.random.default_rng(16)
    page, heads = 64, 8
    stride = ref.page_stride(page, heads)
    pages = (1 << 32) // stride + 40
    pool = torch.zeros(pages, stride, dtype=torch.uint8, device="cuda")
    few = ref.make_pool(rng, 8, page, heads)
    pool[pages - 8:] = _dev(few)
    bt = np.arange(pages - 8, pages, dtype=np.int32)[None]
    q, q64 = _bf16(rng.standard_normal((1, 16, 128)))
    out, lse = B.idx_paged_kv4_attention(q, pool, page, heads, _dev(bt), _dev(np.array([512], np.int32)), 1, SCALE, 512)
    _clean()
    _check_rows(out, lse, q64, few, page, heads, [np.arange(512)])


# ---------------------------------------------------------------------- weights


@pytest.mark.parametrize("page", [64, 16, 100])
@pytest.mark.parametrize("ctx,next_n,heads,group", [([1], 1, 1, 1), ([0, 40, 700], 2, 2, 4), ([513], 4, 1, 20), ([300, 129], 1, 3, 8)])
def test_weights(ctx, next_n, heads, group, page):
    rng = np.random.default_rng(sum(ctx) + group)
    bt, pages, _ = _table(rng, ctx, page)
    pool = ref.make_pool(rng, pages, page, heads)
    width = bt.shape[1] * page + 30
    q, q64 = _bf16(rng.standard_normal((len(ctx) * next_n, heads * group, 128)) * 2)
    ends = [max(0, c - next_n + 1 + j) for c in ctx for j in range(next_n)]
    args = (q, _dev(pool), page, heads, _dev(bt), _dev(np.array(ctx, np.int32)), next_n, SCALE, bt.shape[1] * page)
    _, lse = B.idx_paged_kv4_attention(*args)
    lse = torch.stack([lse.t(), lse.t()], 1)[:, 0].t()  # any strides
    wide = torch.rand(len(ctx), heads, width + 2, device="cuda")
    mass = wide[:, :, 1:-1]
    before = _np(mass)
    want, most = np.zeros(before.shape), 0.0
    for r, e in enumerate(ends):
        for h in range(heads):
            if e == 0:
                continue
            k, v = ref.read(pool, page, heads, _slots(bt, r // next_n, e, page), h)
            hs = slice(h * group, (h + 1) * group)
            s = q64[r, hs] @ k.T * SCALE
            want[r // next_n, h, :e] += np.exp(s - _np(lse[r, hs])[:, None]).sum(0)
            most = max(most, (np.abs(q64[r, hs]) @ np.abs(k).T).max() * SCALE)
    # each weight by its score's error (136 * 2^-23 of its products) and the exponential's, sums
    # of up to next_n * group of them
    ds = 136 * 2.0 ** -23 * most + 2.0 ** -20 + next_n * group * 2.0 ** -24

    def near(got, base):
        assert (np.abs(got - base - want) <= 1.1 * ds * want + 2.0 ** -23 * (base + want)).all()

    out = torch.full_like(wide, 5.0)[:, :, 1:-1]
    got = B.idx_paged_kv4_weights(*args, lse, mass, out)
    _clean()
    assert got.data_ptr() == out.data_ptr()
    near(_np(out), before)
    fresh = B.idx_paged_kv4_weights(*args, lse)
    near(np.pad(_np(fresh), ((0, 0), (0, 0), (0, 30))), 0 * before)
    edges = wide[:, :, [0, -1]].clone()
    assert B.idx_paged_kv4_weights(*args, lse, mass).data_ptr() == mass.data_ptr()
    _clean()
    assert torch.equal(mass, out) and torch.equal(wide[:, :, [0, -1]], edges)


def test_weights_of_what_is_not_finite():
    rng = np.random.default_rng(20)
    bt, pages, _ = _table(rng, [100], 64)
    pool = ref.make_pool(rng, pages, 64, 1)
    slots = _slots(bt, 0, 100, 64)
    (b, _) = ref.spans(64, 1, 0, slots[99] % 64)[2]
    pool[slots[99] // 64, b] = 255
    q, _ = _bf16(rng.standard_normal((2, 3, 128)))
    args = (q, _dev(pool), 64, 1, _dev(bt), _dev(np.array([100], np.int32)), 2, SCALE, 128)
    lse = torch.full((2, 3), 2.0, device="cuda")
    got = B.idx_paged_kv4_weights(*args, lse)
    _clean()
    # the last row alone sees the last token
    assert torch.isfinite(got[..., :99]).all() and torch.isnan(got[..., 99]).all() and (got[..., 100:] == 0).all()


# --------------------------------------------------------------------- eviction


def _evict_reference(mass, ctx, budget, recent, whole):
    nb, heads, _ = mass.shape
    lists = 1 if whole else heads
    keep = np.full((nb, lists, budget), -1, np.int32)
    for b, n in enumerate(ctx):
        kept, last = min(n, budget), min(n, recent)
        for g in range(lists):
            m = mass[b, :, :n].astype(np.float64)
            s = (m.sum(0) if whole else m[g]).astype(np.float32)
            s = np.where(np.isnan(s), np.float32(-3.4028235e38), np.clip(s, np.float32(-3.4028235e38), np.float32(3.4028235e38)))
            old = np.lexsort((np.arange(n - last), -s[:n - last].astype(np.float64)))[:kept - last]
            keep[b, g, :kept] = np.concatenate([np.sort(old), np.arange(n - last, n)])
    return keep


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("ctx,budget,recent,heads,page", [
    ([1], 1, 0, 1, 64), ([5, 0, 64], 8, 3, 2, 16), ([300, 200, 77], 100, 100, 3, 64), ([300, 200, 77], 100, 0, 2, 1),
    ([1000, 3, 513], 250, 17, 4, 48), ([40], 0, 0, 2, 16), ([9000, 8500], 1111, 64, 2, 64)])
def test_evict(whole, ctx, budget, recent, heads, page):
    rng = np.random.default_rng(sum(ctx) + budget)
    new = -(-budget // page)
    bt, pages, spare = _table(rng, ctx, page, new * len(ctx))
    pool0 = ref.make_pool(rng, pages, page, heads, 32)
    columns = max(ctx) + 7
    mass = rng.integers(0, 50, (len(ctx), heads, columns)).astype(np.float32)  # ties among them
    mass[0, 0, :2] = np.nan, np.inf
    wide = _dev(np.concatenate([mass, mass], 2))
    pool, nt = _dev(pool0), spare.reshape(len(ctx), new)
    keep, lens, got = B.idx_kv4_evict(wide[:, :, :columns], _dev(np.array(ctx, np.int32)), budget, recent, pool, page,
                                      _dev(bt), _dev(nt), whole_tokens=whole)
    _clean()
    want = _evict_reference(mass, ctx, budget, recent, whole)
    assert np.array_equal(keep.cpu().numpy(), want)
    assert lens.tolist() == [min(n, budget) for n in ctx]
    moved = pool0.copy()
    for b in range(len(ctx)):
        for h in range(heads):
            for j, t in enumerate(want[b, 0 if whole else h]):
                if t < 0:
                    assert got[b, h, j] == 0
                    continue
                x = mass[b, h, t]
                assert got[b, h, j] == x or np.isnan(x)
                for (a, n), (c, _) in zip(ref.spans(page, heads, h, t % page), ref.spans(page, heads, h, j % page)):
                    moved[nt[b, j // page], c:c + n] = pool0[bt[b, t // page], a:a + n]
    assert np.array_equal(pool.cpu().numpy(), moved)


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("columns,batch,recent", [(262144, 1, 0), (262148, 1, 5), (300001, 2, 64), (9001, 40, 64)])
def test_evict_from_long_contexts(whole, columns, batch, recent):
    """Lists that a cluster just holds, longer ones, and more of them than fit the SMs at once."""
    rng = np.random.default_rng(columns)
    page, heads, budget = 64, 2, 700
    ctx = [columns - 3 * i for i in range(batch)]
    new = -(-budget // page)
    blocks = -(-columns // page)
    # all sequences share the old pages
    bt = np.tile(rng.permutation(blocks).astype(np.int32), (batch, 1))
    nt = (blocks + np.arange(batch * new, dtype=np.int32)).reshape(batch, new)
    pool = torch.zeros(blocks + batch * new, ref.page_stride(page, heads), dtype=torch.uint8, device="cuda")
    mass = rng.random((batch, heads, columns), dtype=np.float32)
    mass[:, :, ::3] = 0.75  # ties
    keep, lens, got = B.idx_kv4_evict(_dev(mass), _dev(np.array(ctx, np.int32)), budget, recent, pool, page, _dev(bt),
                                      _dev(nt), whole_tokens=whole)
    _clean()
    assert np.array_equal(keep.cpu().numpy(), _evict_reference(mass, ctx, budget, recent, whole))
    want = np.take_along_axis(mass, np.broadcast_to(keep.cpu().numpy().astype(np.int64), (batch, heads, budget)), 2)
    assert np.array_equal(got.cpu().numpy(), want) and lens.tolist() == [budget] * batch


def test_evict_past_the_columns_and_the_pool():
    pool = torch.ones(6, ref.page_stride(16, 1), dtype=torch.uint8, device="cuda")
    mass = torch.rand(2, 1, 40, device="cuda")
    bt = torch.tensor([[0, 1, 2], [0, 9, 1]], dtype=torch.int32, device="cuda")
    nt = torch.tensor([[3], [4]], dtype=torch.int32, device="cuda")
    keep, lens, _ = B.idx_kv4_evict(mass, torch.tensor([50, 10], dtype=torch.int32, device="cuda"), 12, 2, pool, 16, bt, nt)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_BOUNDS
    assert lens.tolist() == [12, 10] and keep[0, 0, -2:].tolist() == [38, 39]
    keep, lens, _ = B.idx_kv4_evict(mass, torch.tensor([12, 40], dtype=torch.int32, device="cuda"), 12, 12, pool, 16, bt,
                                    torch.tensor([[6], [4]], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_PAGE
    # positions 28 to 31 of the second lie on no page: zeros
    assert (pool[4, :4 * 64] == 0).all() and (pool[4, 4 * 64:12 * 64] == 1).all()


# ---------------------------------------------------------------------- prefill


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (3, 5), (1, 16)])
@pytest.mark.parametrize("lens", [[(1, 1)], [(0, 5), (65, 65), (7, 300)], [(128, 128), (129, 0), (300, 200)],
                                  [(257, 700), (3, 3), (1, 129)]])
def test_prefill(lens, heads, group, causal):
    rng = np.random.default_rng(sum(a + 3 * b for a, b in lens) + heads)
    nq, nk = sum(a for a, _ in lens), sum(b for _, b in lens)
    q, q64 = _bf16(rng.standard_normal((nq + 2, heads * group, 136)) * 2)
    kv, kv64 = _bf16(rng.standard_normal((nk, 2, heads, 128)))
    cq = np.concatenate([[0], np.cumsum([a for a, _ in lens])]).astype(np.int32)
    ck = np.concatenate([[0], np.cumsum([b for _, b in lens])]).astype(np.int32)
    out = torch.full((nq + 2, heads * group, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((nq + 2, heads * group), 9.0, device="cuda")
    B.idx_grouped_prefill(q[:, :, :128], kv[:, 0], kv[:, 1], _dev(cq), _dev(ck), SCALE, causal=causal, out=out, lse=lse)
    _clean()
    assert (out[nq:] == 9).all() and (lse[nq:] == 9).all()
    for b, (a, m) in enumerate(lens):
        seen = np.tril(np.ones((a, m), bool), m - a) if causal else None
        rows = slice(cq[b], cq[b + 1])
        for h in range(heads * group):
            k, v = kv64[ck[b]:ck[b + 1], 0, h // group], kv64[ck[b]:ck[b + 1], 1, h // group]
            ref.check(_np(out[rows, h]), _np(lse[rows, h]), ref.attend(q64[rows, h, :128], k, v, SCALE, seen), m,
                      ref.HALF_BF16, 1e-3)


def test_prefill_long_rows_are_cut_and_joined():
    rng = np.random.default_rng(30)
    q, q64 = _bf16(rng.standard_normal((40, 6, 128)))
    k, k64 = _bf16(rng.standard_normal((20000, 2, 128)))
    v, v64 = _bf16(rng.standard_normal((20000, 2, 128)))
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = B.idx_grouped_prefill(q, k, v, cu(40), cu(20000), SCALE)
    _clean()
    seen = np.tril(np.ones((40, 20000), bool), 19960)
    for h in range(6):
        ref.check(_np(out[:, h]), _np(lse[:, h]), ref.attend(q64[:, h], k64[:, h // 3], v64[:, h // 3], SCALE, seen), 20000,
                  ref.HALF_BF16, 1e-4)
