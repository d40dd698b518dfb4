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


@pytest.mark.parametrize("rows", [3, 20, 300])
def test_short_lists_that_descend(rows):
    """A list of few slots whose bounds descend is told of and left alone like a long one."""
    rng = np.random.default_rng(rows)
    pool = ref.make_pool(rng, 8, 64, 1)
    slots = rng.integers(0, 512, 500)
    q, q64 = _bf16(rng.standard_normal((rows, 2, 128)))
    out = torch.full((rows, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, 2), 5.0, device="cuda")
    args = (q, _dev(pool), 64, 1, _dev(slots.astype(np.int32)))
    bounds = np.array(([0, 500] * rows)[:rows + 1], np.int32)
    listed = sum(max(1, -(-int(b - a) // 128)) for a, b in zip(bounds, bounds[1:]))
    assert listed > 500 // 128 + rows
    B.idx_kv4_attention(*args, _dev(bounds), SCALE, out=out, lse=lse)
    assert _status() == B.DEV_BAD_BOUNDS and (out == 5).all() and (lse == 5).all()
    # one that ascends, full and clipped rows among its rows, is computed
    cuts = np.sort(rng.integers(0, 500, rows - 1))
    bounds = np.concatenate([[-7], cuts, [900]]).astype(np.int32)
    B.idx_kv4_attention(*args, _dev(bounds), SCALE, out=out, lse=lse)
    _clean()
    cut = np.clip(bounds, 0, 500)
    _check_rows(out, lse, q64, pool, 64, 1, [slots[a:b] for a, b in zip(cut, cut[1:])])


@pytest.mark.parametrize("factor,scale", [(1e-37, 1e-12), (1e-37, 1e-39), (1.0, 1e-40), (1e30, 1e-45), (0.0, 1e-12)])
@pytest.mark.parametrize("n", [40, 700])
def test_factors_whose_product_leaves_the_range(factor, scale, n):
    """Queries and factors so small that every score is zero: tokens that are there weigh alike,
    those that are not weigh nothing."""
    rng = np.random.default_rng(n)
    bt, pages, _ = _table(rng, [n], 64)
    pool = ref.make_pool(rng, pages, 64, 2)
    slots = _slots(bt, 0, n, 64)
    q, q64 = _bf16(rng.choice([-1.0, 1.0], (2, 8, 128)) * factor)
    ctx = _dev(np.array([n], np.int32))
    paged = (q, _dev(pool), 64, 2, _dev(bt), ctx, 2, scale, n)
    out, lse = B.idx_paged_kv4_attention(*paged)
    weights = B.idx_paged_kv4_weights(*paged, lse)
    listed, ll = B.idx_kv4_attention(q[1:], _dev(pool), 64, 2, _dev(slots.astype(np.int32)), _dev(np.array([0, n], np.int32)),
                                     scale)
    _clean()
    for h in range(2):
        k, v = ref.read(pool, 64, 2, slots, h)
        hs = slice(4 * h, 4 * h + 4)
        for j in range(2):
            m = n - 1 + j
            want = ref.attend(q64[j, hs], k[:m], v[:m], float(np.float32(scale)))
            ref.check(_np(out[j, hs]), _np(lse[j, hs]), want, m, vmax=np.abs(v).max())
        ref.check(_np(listed[0, hs]), _np(ll[0, hs]), want, n, vmax=np.abs(v).max())
        # each weight is 1 / m by at most the errors of its logarithm and its exponential, and of
        # sums of eight
        got = _np(weights[0, h])
        wish = np.full(n, 4 / n)
        wish[:n - 1] += 4 / (n - 1)
        assert (np.abs(got - wish) <= wish * (2.0 ** -19 + 2.0 ** -21 * np.log(n))).all()


@pytest.mark.parametrize("n", [300, 700, 9000])
@pytest.mark.parametrize("bits", [2, 9])
def test_values_near_the_least(n, bits):
    """Values near the least that 32 bits hold come out as they are, not as zeros."""
    rng = np.random.default_rng(n + bits)
    bt, pages, _ = _table(rng, [n], 64)
    pool = ref.make_pool(rng, pages, 64, 1)
    m = 64
    pool[:, m * 132:m * 136] = rng.integers(bits - 2, bits + 3, (pages, m * 4)).astype(np.uint8)
    q, q64 = _bf16(rng.standard_normal((1, 8, 128)))
    out, _ = B.idx_paged_kv4_attention(q, _dev(pool), 64, 1, _dev(bt), _dev(np.array([n], np.int32)), 1, SCALE, n)
    _clean()
    k, v = ref.read(pool, 64, 1, _slots(bt, 0, n, 64), 0)
    o, _, pv, mag = ref.attend(q64[0], k, v, SCALE)
    # the bounds of kv4_ref.check; sums in 32 bits' least steps (2^-149) a token and a joining, the
    # result in bf16's (2^-133)
    ds = 136 * 2.0 ** -23 * mag + 2.0 ** -20
    tol = (ref.HALF_BF16 * np.abs(o) + (ref.HALF_F16 * 1.01 + 2 * ds[:, None]) * pv * (1 + ref.HALF_BF16)
           + n * 2.0 ** -26 * np.abs(v).max() + 64 * 2.0 ** -149 + 2.0 ** -134)
    assert (np.abs(_np(out[0]) - o) <= tol).all()
    assert np.abs(o).max() > 8 * tol.max()  # (zeros would show)


# ------------------------------------------------------ shares of several tiles


@pytest.mark.parametrize("page", [64, 100])
@pytest.mark.parametrize("group,next_n", [(1, 1), (4, 2), (40, 1)])
@pytest.mark.parametrize("bad", [False, True])
def test_shares_of_several_tiles(page, group, next_n, bad):
    """Lists with several times more tiles than shares, sequences that end inside shares, pages
    outside the pool among them; weights into a tensor of their own and in place."""
    rng = np.random.default_rng(page + group + bad)
    heads = 8
    ctx = [0, 1, 63] + [int(x) for x in rng.integers(3000, 9001, 12)]
    bt, pages, _ = _table(rng, ctx, page)
    pool = ref.make_pool(rng, pages, page, heads)
    slots = [_slots(bt, b, n, page) for b, n in enumerate(ctx)]
    wrong, there = bt.copy(), [np.ones(n, bool) for n in ctx]
    if bad:
        for b in (4, 9):
            for at, p in ((0, -1), (17, pages), (ctx[b] // page, -5)):
                wrong[b, at] = p
                there[b][at * page:(at + 1) * page] = False
    q, q64 = _bf16(rng.standard_normal((len(ctx) * next_n, heads * group, 128)))
    longest = bt.shape[1] * page
    args = (q, _dev(pool), page, heads, _dev(wrong), _dev(np.array(ctx, np.int32)), next_n, SCALE, longest)
    out, lse = B.idx_paged_kv4_attention(*args)
    wide = torch.rand(len(ctx), heads, longest + 5, device="cuda")
    mass = wide[:, :, 2:-2]
    before = _np(mass)
    own = torch.full_like(wide, 7.0)[:, :, 2:-2]
    B.idx_paged_kv4_weights(*args, lse, mass, own)
    edges = wide[:, :, [0, 1, -2, -1]].clone()
    B.idx_paged_kv4_weights(*args, lse, mass)
    assert _status() == (B.DEV_BAD_PAGE if bad else 0)
    assert torch.equal(mass, own) and torch.equal(wide[:, :, [0, 1, -2, -1]], edges)
    got, blocks = _np(own), -(-group * next_n // 32)
    # each page is read through kv4_ref once a sampled head
    for b, h in [(0, 0), (1, 5), (2, 7), (3, 0), (4, 3), (9, 7), (9, 2), (14, 7)]:
        k, v = ref.read(pool, page, heads, slots[b], h)
        hs = slice(h * group, (h + 1) * group)
        want, most = np.zeros(longest + 1), 0.0
        for j in range(next_n):
            r, end = b * next_n + j, max(0, ctx[b] - next_n + 1 + j)
            seen = there[b][:end]
            ref.check(_np(out[r, hs]), _np(lse[r, hs]), ref.attend(q64[r, hs], k[:end][seen], v[:end][seen], SCALE), end,
                      vmax=np.abs(v).max() if v.size else 0)
            if seen.any():
                s = q64[r, hs] @ k[:end].T * SCALE
                want[:end] += np.where(seen, np.exp(s - _np(lse[r, hs])[:, None]), 0).sum(0)
                most = max(most, (np.abs(q64[r, hs]) @ np.abs(k).T).max() * SCALE)
        # as for short contexts, and a rounding of the sum so far for each block of columns
        ds = 136 * 2.0 ** -23 * most + 2.0 ** -20 + next_n * group * 2.0 ** -24
        base = before[b, h]
        assert (np.abs(got[b, h] - base - want) <= 1.1 * ds * want + (blocks + 1) * 2.0 ** -24 * (base + want)).all(), (b, h)


@pytest.mark.parametrize("page", [64, 100])
def test_teams_of_several_steps(page):
    """Few long contexts, which clusters share, several tiles a group."""
    rng = np.random.default_rng(page)
    ctx, heads = [9000, 7001], 2
    assert B.kv4_attention_workspace_size(4, 16, heads, 9000, next_n=2) == 0
    bt, pages, _ = _table(rng, ctx, page)
    pool = ref.make_pool(rng, pages, page, heads)
    q, q64 = _bf16(rng.standard_normal((4, 16, 128)))
    out, lse = B.idx_paged_kv4_attention(q, _dev(pool), page, heads, _dev(bt), _dev(np.array(ctx, np.int32)), 2, SCALE, 9000)
    _clean()
    _check_rows(out, lse, q64, pool, page, heads, [_slots(bt, b, n, page)[:n - 1 + j] for b, n in enumerate(ctx) for j in (0, 1)])


@pytest.mark.parametrize("page", [64, 48])
def test_weights_with_a_length_for_each_row(page):
    """Rows of one sequence that see more, fewer and none of its tokens, past the limit among them."""
    rng = np.random.default_rng(page)
    bt, pages, _ = _table(rng, [900, 700], page)
    pool = ref.make_pool(rng, pages, page, 2)
    q, q64 = _bf16(rng.standard_normal((6, 8, 128)))
    per, most = np.array([900, 3, 0, 650, 700, -2], np.int32), 800
    args = (q, _dev(pool), page, 2, _dev(bt), _dev(per), 3, SCALE, most)
    _, lse = B.idx_paged_kv4_attention(*args, ctx_per_row=True)
    got = B.idx_paged_kv4_weights(*args, lse, ctx_per_row=True)
    _clean()
    want, mag = np.zeros((2, 2, most)), 0.0
    for r, end in enumerate(np.clip(per, 0, most)):
        for h in range(2):
            if end:
                k, _ = ref.read(pool, page, 2, _slots(bt, r // 3, end, page), h)
                hs = slice(4 * h, 4 * h + 4)
                want[r // 3, h, :end] += np.exp(q64[r, hs] @ k.T * SCALE - _np(lse[r, hs])[:, None]).sum(0)
                mag = max(mag, (np.abs(q64[r, hs]) @ np.abs(k).T).max() * SCALE)
    # each weight by its score's and its exponential's errors, sums of twelve
    ds = 136 * 2.0 ** -23 * mag + 2.0 ** -20 + 12 * 2.0 ** -24
    assert (np.abs(_np(got) - want) <= 1.1 * ds * want + 2.0 ** -23 * want).all()


# --------------------------------------------------------------- eviction's order


def _evicted(mass, budget, recent, whole):
    """keep [B, lists, budget] of whole contexts on one page a token, which nothing depends on."""
    nb, heads, n = mass.shape
    page = 4096
    blocks, new = -(-n // page), -(-budget // page)
    pool = torch.zeros(blocks + nb * new, ref.page_stride(page, heads), dtype=torch.uint8, device="cuda")
    bt = torch.arange(blocks, dtype=torch.int32, device="cuda").expand(nb, blocks).contiguous()
    nt = (blocks + torch.arange(nb * new, dtype=torch.int32, device="cuda")).view(nb, new)
    ctx = torch.full((nb,), n, dtype=torch.int32, device="cuda")
    keep, _, _ = B.idx_kv4_evict(mass, ctx, budget, recent, pool, page, bt, nt, whole_tokens=whole)
    _clean()
    return keep.cpu().numpy()


@pytest.mark.parametrize("columns", [37, 300, 2500, 9003, 262149])
@pytest.mark.parametrize("whole", [False, True])
def test_zeros_of_either_sign_weigh_alike(columns, whole):
    rng = np.random.default_rng(columns)
    heads = 2
    mass = np.where(rng.random((2, heads, columns)) < 0.5, -0.0, 0.0).astype(np.float32)
    budget = min(columns // 2, 1000)
    keep = _evicted(_dev(mass), budget, 3, whole)
    want = np.concatenate([np.arange(budget - 3), np.arange(columns - 3, columns)])
    assert (keep == want).all()


@pytest.mark.parametrize("columns", [37, 300, 2500, 9003, 262149])
@pytest.mark.parametrize("whole", [False, True])
def test_infinities_count_as_the_largest_numbers(columns, whole):
    """As the header says: infinities as the largest and the least float, NaN as the least."""
    rng = np.random.default_rng(columns + 1)
    most = np.float32(3.4028235e38)
    x = rng.choice(np.array([np.inf, most, 1, 0, -1, -most, -np.inf, np.nan], np.float32), columns)
    mass = np.zeros((1, 2, columns), np.float32)
    mass[0, 0] = x
    mass[0, 1] = 0 if whole else x
    budget = min(columns // 2, 1500)
    keep = _evicted(_dev(mass), budget, 0, whole)
    y = np.clip(np.where(np.isnan(x), -most, x), -most, most).astype(np.float64)
    assert (keep == np.sort(np.lexsort((np.arange(columns), -y))[:budget])).all()


@pytest.mark.parametrize("heads", [3, 5, 8, 11])
@pytest.mark.parametrize("columns", [300, 2048, 9003, 262149])
def test_sums_over_heads_are_rounded_once(heads, columns):
    """Tokens whose heads share the same weights in different orders have one sum, and one bit more
    in a head's weight counts: sums in 32 bits would part the first and miss the second.  (Weights
    are multiples of 2^-30 below 1: their sums are exact in 64 bits and in pairs of floats.)"""
    rng = np.random.default_rng(heads * columns)
    one = rng.integers(1, 1 << 24, heads) * 2.0 ** -30
    one[0] = 0.75 + 2.0 ** -24
    mass = rng.permuted(np.tile(one, (columns, 1)), axis=1).T.astype(np.float32)[None]
    ulp = np.spacing(np.float32(one.sum()))
    heavy = rng.random(columns) < 0.1
    mass[0, :, heavy] = one
    for t in np.flatnonzero(heavy):  # the least weight more by the sum's own step
        mass[0, -1, t] = np.float32(one[-1] + ulp)
    total = mass[0].astype(np.float64).sum(0).astype(np.float32)
    assert len(np.unique(total)) == 2 and (total[heavy] > total[~heavy].max()).all()
    for budget in (min(heavy.sum() // 2, 1000), min(heavy.sum() + columns // 3, 4000)):
        want = np.sort(np.lexsort((np.arange(columns), -total.astype(np.float64)))[:budget])
        assert (_evicted(_dev(mass), int(budget), 0, True) == want).all()


# ------------------------------------------------------------- written views


def test_views_beside_one_another():
    """Sums and read-back rows that share storage, not elements, and outputs whose heads are
    outermost; views that share elements are refused before anything is launched."""
    rng = np.random.default_rng(60)
    page, heads, ctx = 64, 2, [70, 300]
    bt, pages, _ = _table(rng, ctx, page)
    pool = _dev(ref.make_pool(rng, pages, page, heads))
    lens = _dev(np.array(ctx, np.int32))
    q, _ = _bf16(rng.standard_normal((2, 8, 128)))
    paged = (q, pool, page, heads, _dev(bt), lens, 1, SCALE, 320)
    out, lse = B.idx_paged_kv4_attention(*paged)
    turned = torch.zeros(8, 2, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    B.idx_paged_kv4_attention(*paged, out=turned)
    mass = torch.rand(2, heads, 330, device="cuda")
    want = B.idx_paged_kv4_weights(*paged, lse, mass, torch.empty_like(mass))
    for shape, at in [((2, 2, heads, 330), lambda t, i: t[:, i]), ((2, heads, 2, 330), lambda t, i: t[:, :, i]),
                      ((2, heads, 660), lambda t, i: t[..., 330 * i:330 * i + 330]),
                      ((heads, 2, 2, 330), lambda t, i: t[:, i].transpose(0, 1))]:
        both = torch.zeros(shape, device="cuda")
        for i in (0, 1):
            both.zero_()
            at(both, i).copy_(mass)
            got = B.idx_paged_kv4_weights(*paged, lse, at(both, i), at(both, 1 - i))
            assert torch.equal(got, want) and torch.equal(at(both, i), mass)
    # one row of sums read for all heads, written elsewhere
    one = mass[:, :1].expand(2, heads, 330)
    assert torch.equal(B.idx_paged_kv4_weights(*paged, lse, one, torch.empty_like(mass)),
                       B.idx_paged_kv4_weights(*paged, lse, one.contiguous()))
    cu = _dev(np.array([0, 70, 370], np.int32))
    rows = [torch.zeros(370, heads, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    B.idx_kv4_gather(pool, page, _dev(bt), cu, *rows)
    for shape, at in [((370, heads, 2, 128), lambda t, i: t[:, :, i]), ((370, 2, heads, 128), lambda t, i: t[:, i]),
                      ((2, heads, 370, 128), lambda t, i: t[i].transpose(0, 1)), ((heads, 370, 256), lambda t, i: t.transpose(0, 1)[..., 128 * i:128 * i + 128])]:
        both = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        B.idx_kv4_gather(pool, page, _dev(bt), cu, at(both, 0), at(both, 1))
        assert torch.equal(at(both, 0), rows[0]) and torch.equal(at(both, 1), rows[1])
    _clean()
    assert torch.equal(turned, out)
    wide, held = torch.zeros(2, heads, 331, device="cuda"), torch.zeros(2, 1, 330, device="cuda")
    spot = torch.zeros(370, 1, 128, dtype=torch.bfloat16, device="cuda")
    new = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    for call in [lambda: B.idx_paged_kv4_weights(*paged, lse, held.expand(2, heads, 330)),
                 lambda: B.idx_paged_kv4_weights(*paged, lse, mass, held.expand(2, heads, 330)),
                 lambda: B.idx_paged_kv4_weights(*paged, lse, wide[..., :-1], wide[..., 1:]),
                 lambda: B.idx_paged_kv4_attention(*paged, out=spot[:2].expand(2, 8, 128)),
                 lambda: B.idx_kv4_gather(pool, page, _dev(bt), cu, spot.expand(370, heads, 128), rows[1]),
                 lambda: B.idx_kv4_gather(pool, page, _dev(bt), cu, rows[0], rows[0]),
                 lambda: B.idx_kv4_evict(mass, lens, 60, 4, pool, page, _dev(bt), new, new_lens=lens),
                 lambda: B.idx_kv4_evict(mass, lens, 330, 4, pool, page, _dev(bt), new.expand(2, 6).contiguous(), new_mass=mass)]:
        with pytest.raises(B.IndexerError, match="INVALID"):
            call()
    torch.cuda.synchronize()
    assert lens.tolist() == ctx and not wide.any() and not held.any() and not spot.any()
