"""GPU parity of the latent cache and its attention with plain 64-bit
statements (latent_ref), at the lengths, head counts, strides and slots where
the kernels' tiles end, and with everything outside the rows poisoned."""
import numpy as np
import pytest
import torch

import latent_ref as ref
from sparse_attention_indexer_mxfp4_gb300 import _binding as B

pytestmark = pytest.mark.gpu
FMTS = [ref.BF16, ref.FP8]
SCALE = 192 ** -0.5


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


# ------------------------------------------------------------------------ store


def _store_reference(x, pos, cs, w, eps):
    y = x[:, :ref.L]
    if w is not None:
        y = y / np.sqrt((y * y).mean(1, keepdims=True) + eps) * w
    r = x[:, ref.L:]
    if cs is not None:
        c, s = cs[pos][:, :32], cs[pos][:, 32:64]
        r = np.stack([r[:, ::2] * c - r[:, 1::2] * s, r[:, 1::2] * c + r[:, ::2] * s], -1).reshape(len(x), 64)
    return y, r


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tokens,page,extra", [(1, 64, 0), (5, 1, 16), (67, 48, 32), (300, 64, 0), (3001, 16, 0)])
@pytest.mark.parametrize("norm,rope", [(True, True), (False, True), (True, False)])
def test_store(fmt, tokens, page, extra, norm, rope):
    rng = np.random.default_rng(tokens + page)
    pages = -(-tokens // page) + 3
    kv = rng.standard_normal((tokens, 640)) * np.exp(2 * rng.standard_normal((tokens, 1)))
    kv[0, :130] = 0  # groups of zeros
    t, x = _bf16(kv)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    slots[tokens // 2] = -1 if tokens > 1 else slots[0]
    cs = rng.standard_normal((50, 72)).astype(np.float32)
    pos = rng.integers(0, 50, tokens).astype(np.int32)
    w = (1 + 0.1 * rng.standard_normal(ref.L)).astype(np.float32)
    pool0 = rng.integers(0, 256, (pages, ref.page_stride(fmt, page, extra)), dtype=np.uint8)
    pool = _dev(pool0)
    B.idx_latent_store(t[:, :576], _dev(pos) if rope else None, _dev(cs) if rope else None,
                       _dev(w) if norm else None, 1e-6, pool, page, _dev(slots), fmt)
    _clean()
    got = pool.cpu().numpy()
    y, r = _store_reference(x[:, :576], pos, cs.astype(np.float64) if rope else None,
                            w.astype(np.float64) if norm else None, 1e-6)
    live = slots >= 0
    read = ref.read_tokens(got, fmt, page, slots[live])
    y, r = y[live], r[live]
    # 32-bit arithmetic before the rounding: a few units of 2^-22
    rtol = ref.HALF_BF16 + 2.0 ** -20
    rmag = np.repeat(np.abs(r).reshape(-1, 32, 2).max(-1), 2, 1)  # a rotation may cancel
    assert (np.abs(read[:, ref.L:] - r) <= ref.HALF_BF16 * np.abs(r) + 2.0 ** -18 * (rmag + 1)).all()
    if fmt == ref.BF16:
        assert (np.abs(read[:, :ref.L] - y) <= rtol * np.abs(y) + 1e-37).all()
    else:
        amax = np.abs(y).reshape(-1, 8, 64).max(-1)
        exact = np.log2(np.maximum(amax, 2.0 ** -126) / 448)
        want = np.clip(np.ceil(exact) + 127, 0, 254)
        s = slots[live]
        bits = np.stack([got[a // page][page * 640 + (a % page) * 8:][:8] for a in s]).astype(int)
        near = np.abs(exact - np.round(exact)) < 1e-5
        assert ((bits == want) | (near & (np.abs(bits - want) == 1))).all()
        step = np.repeat(2.0 ** (bits - 127.0), 64, 1)
        # e4m3: half a step is 2^-4 of the value, 2^-10 below the normal range
        assert (np.abs(read[:, :ref.L] - y) <= (2.0 ** -4 + 1e-5) * np.abs(y) + (2.0 ** -10 + 1e-5) * step).all()
    # nothing else is touched
    back = got.copy()
    tb = ref.token_bytes(fmt)
    for a in slots[live]:
        p, o = a // page, a % page
        spans = [(o * tb, tb)] if fmt == ref.BF16 else [
            (o * 512, 512), (page * 512 + o * 128, 128), (page * 640 + o * 8, 8)]
        for at, n in spans:
            back[p, at:at + n] = pool0[p, at:at + n]
    assert np.array_equal(back, pool0)


def test_store_codes_are_nearest():
    """Codes of values around every e4m3 midpoint, with the group's exponent pinned at 0."""
    grid = ref.e4m3_float(np.arange(0x7f, dtype=np.uint8))
    x = np.concatenate([grid, (grid[1:] + grid[:-1]) / 2, -(grid[1:] + grid[:-1]) / 2, -grid])[:448]
    kv = np.zeros((1, 576))
    kv[0, :448].reshape(7, 64)[:] = x.reshape(7, 64)
    kv[0, :448:64] = 448.0
    t, v = _bf16(kv)
    pool = torch.zeros(1, 648 * 2, dtype=torch.uint8, device="cuda")
    B.idx_latent_store(t, None, None, None, 0.0, pool, 2, _dev(np.array([1], np.int64)), ref.FP8)
    _clean()
    want = torch.from_numpy(v[0, :512].astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(pool.cpu().numpy()[0, 512:1024], want)


def test_store_not_finite_and_bad_places():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 576))
    x[1, 70], x[2, 200] = np.nan, np.inf
    t, v = _bf16(x)
    pool = torch.zeros(2, 64 * 648, dtype=torch.uint8, device="cuda")
    cs = torch.ones(4, 64, device="cuda")
    pos = torch.tensor([0, 1, 2, 3, 4, -1], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 1, 2, 128, 4, 5], device="cuda")
    B.idx_latent_store(t, pos, cs, None, 0.0, pool, 64, slots, ref.FP8)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_PAGE | B.DEV_BAD_POSITION
    got = ref.read_tokens(pool.cpu().numpy(), ref.FP8, 64, np.arange(6))
    assert np.isnan(got[1, 64:128]).all() and np.isfinite(got[1, :64]).all()
    assert np.isnan(got[2, 192:256]).all() and np.isfinite(got[2, 256:512]).all()
    assert (np.abs(got[0, :512] - v[0, :512]) <= 2.0 ** -4 * np.abs(v[0, :512]) + 2.0 ** -10).all()
    assert (got[3:] == 0).all()


# ----------------------------------------------------------------------- gather


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,page", [([1], 64), ([0, 5, 0, 130, 1], 16), ([64, 63, 65], 64), ([7, 0], 1),
                                       ([2000, 3], 48)])
def test_gather(fmt, lens, page):
    rng = np.random.default_rng(sum(lens) + page)
    start = rng.integers(0, 70, len(lens)).astype(np.int32)
    need = [-(-(int(s) + n) // page) for s, n in zip(start, lens)]
    pages = sum(need) + 2
    pool = ref.make_pool(rng, fmt, pages, page, 32)
    perm = rng.permutation(pages).astype(np.int32)
    bt = np.full((len(lens), max(need) + 1), -5, np.int32)
    at, rows = 0, []
    for b, n in enumerate(lens):
        bt[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        pos = start[b] + np.arange(n)
        rows.append(bt[b, pos // page].astype(np.int64) * page + pos % page)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    N = int(cu[-1])
    out = torch.full((N + 3, 640), 7.0, dtype=torch.bfloat16, device="cuda")
    B.idx_latent_gather(_dev(pool), page, fmt, _dev(bt), _dev(cu), out[:, :576], seq_starts=_dev(start))
    _clean()
    got = _np(out)
    want = ref.read_tokens(pool, fmt, page, np.concatenate(rows))
    assert np.array_equal(got[:N, :576], want)
    assert (got[N:] == 7).all() and (got[:, 576:] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_gather_bad_pages(fmt):
    rng = np.random.default_rng(1)
    pool = ref.make_pool(rng, fmt, 3, 64)
    bt = np.array([[2, 9, -1]], np.int32)
    out = torch.full((256, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    B.idx_latent_gather(_dev(pool), 64, fmt, _dev(bt), _dev(np.array([0, 256], np.int32)), out)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_PAGE
    got = _np(out)
    assert np.array_equal(got[:64], ref.read_tokens(pool, fmt, 64, 128 + np.arange(64))) and (got[64:] == 0).all()


# ------------------------------------------------------------- absorbed attention


def _sparse_case(rng, fmt, lens, H, page, gain=1.0, extra=0):
    total = int(sum(lens))
    pages = -(-max(total, 1) * 2 // page) + 1
    pool = ref.make_pool(rng, fmt, pages, page, extra)
    slots = rng.permutation(pages * page)[:total].astype(np.int32)
    ref.poison(pool, fmt, page, slots)
    indptr = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    qt, q = _bf16(gain * rng.standard_normal((len(lens), H, 576)))
    return pool, slots, indptr, qt, q


def _check_sparse(pool, fmt, page, slots, indptr, q, out, lse, rows=None):
    out, lse = _np(out), None if lse is None else _np(lse)
    for r in range(len(indptr) - 1) if rows is None else rows:
        tok = ref.read_tokens(pool, fmt, page, slots[indptr[r]:indptr[r + 1]])
        ref.check(out[r], None if lse is None else lse[r], ref.attend(q[r], tok, tok[:, :512], SCALE))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H", [1, 3, 8, 16, 17, 32, 40, 64, 65, 96, 128])
@pytest.mark.parametrize("longest", [130, 700])  # rows that stay whole, and a row cut into pieces
def test_sparse_heads(fmt, H, longest):
    rng = np.random.default_rng(H)
    pool, slots, indptr, qt, q = _sparse_case(rng, fmt, [longest, 0, 64, 1], H, 64)
    out, lse = B.idx_latent_attention(qt, _dev(pool), 64, fmt, _dev(slots), _dev(indptr), SCALE)
    _clean()
    _check_sparse(pool, fmt, 64, slots, indptr, q, out, lse)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,page", [([1], 64), ([0], 64), ([2], 1), ([31, 32, 33], 16), ([63, 64, 65, 0], 64),
                                       ([127, 128, 129, 0, 0, 7], 128), ([2048], 64), ([5000, 1, 3], 48),
                                       ([3] * 400, 64), ([191, 193] * 90, 64)])
def test_sparse_lengths(fmt, lens, page):
    rng = np.random.default_rng(sum(lens) + len(lens))
    pool, slots, indptr, qt, q = _sparse_case(rng, fmt, lens, 16, page, extra=16)
    out, lse = B.idx_latent_attention(qt, _dev(pool), page, fmt, _dev(slots), _dev(indptr), SCALE)
    _clean()
    _check_sparse(pool, fmt, page, slots, indptr, q, out, lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_sparse_many_rows_wide(fmt):
    """More (row, head group) pairs than a wave of CTAs holds, uneven lengths."""
    rng = np.random.default_rng(9)
    lens = rng.integers(0, 400, 330)
    pool, slots, indptr, qt, q = _sparse_case(rng, fmt, lens, 128, 64)
    out, lse = B.idx_latent_attention(qt, _dev(pool), 64, fmt, _dev(slots), _dev(indptr), SCALE)
    _clean()
    _check_sparse(pool, fmt, 64, slots, indptr, q, out, lse, rows=list(range(0, 330, 7)) + [329])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gain", [0.0, 20.0])
def test_sparse_flat_and_peaked(fmt, gain):
    """Equal scores, and scores so far apart that the running maximum moves by hundreds."""
    rng = np.random.default_rng(5)
    pool, slots, indptr, qt, q = _sparse_case(rng, fmt, [700, 65], 64, 64, gain)
    tok = ref.read_tokens(pool, fmt, 64, slots[:700])
    slots[:700] = slots[:700][np.argsort(tok @ q[0, 0])]  # head 0's scores rise along the row
    out, lse = B.idx_latent_attention(qt, _dev(pool), 64, fmt, _dev(slots), _dev(indptr), SCALE)
    _clean()
    _check_sparse(pool, fmt, 64, slots, indptr, q, out, lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_sparse_strides_outputs_and_repeats(fmt):
    rng = np.random.default_rng(6)
    pool, slots, indptr, _, _ = _sparse_case(rng, fmt, [100, 70, 0], 24, 64)
    slots[5:9] = slots[4]  # a slot listed again counts again
    big, q = _bf16(rng.standard_normal((3, 30, 584)))
    o = torch.full((3, 30, 520), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 28), 3.0, device="cuda")
    ws = torch.empty(B.latent_attention_workspace_size(3, 24, 300) + 8, dtype=torch.uint8, device="cuda")
    got, gl = B.idx_latent_attention(big[:, 2:26, :576], _dev(pool), 64, fmt, _dev(slots), _dev(indptr), SCALE,
                                     out=o[:, 3:27, :512], lse=lse[:, :24], workspace=ws)
    _clean()
    _check_sparse(pool, fmt, 64, slots, indptr, q[:, 2:26, :576], got, gl)
    assert (o[:, :3] == 3).all() and (o[:, 27:] == 3).all() and (o[..., 512:] == 3).all() and (lse[:, 24:] == 3).all()
    again, none = B.idx_latent_attention(big[:, 2:26, :576], _dev(pool), 64, fmt, _dev(slots), _dev(indptr), SCALE,
                                         lse=False)
    assert none is None and torch.equal(again, got)


@pytest.mark.parametrize("fmt", FMTS)
def test_sparse_bad_slots(fmt):
    """Slots outside the pool are left out; a row of nothing else is empty."""
    rng = np.random.default_rng(7)
    pool, slots, indptr, qt, q = _sparse_case(rng, fmt, [150, 20, 90], 16, 64)
    bad = slots.copy()
    bad[3], bad[70], bad[150:170] = -1, pool.shape[0] * 64, 2 ** 31 - 1
    bad[171] = -7
    out, lse = B.idx_latent_attention(qt, _dev(pool), 64, fmt, _dev(bad), _dev(indptr), SCALE)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_PAGE
    out, lse = _np(out), _np(lse)
    for r in range(3):
        s = bad[indptr[r]:indptr[r + 1]]
        tok = ref.read_tokens(pool, fmt, 64, s[(s >= 0) & (s < pool.shape[0] * 64)])
        ref.check(out[r], lse[r], ref.attend(q[r], tok, tok[:, :512], SCALE))


@pytest.mark.parametrize("fmt", FMTS)
def test_not_finite_tokens_show(fmt):
    """A row that holds a NaN token is NaN; the rows beside it are not."""
    rng = np.random.default_rng(10)
    pool, slots, indptr, qt, q = _sparse_case(rng, fmt, [80, 80, 80], 16, 64)
    ref.poison(pool, fmt, 64, np.delete(slots, 100))
    out, lse = B.idx_latent_attention(qt, _dev(pool), 64, fmt, _dev(slots), _dev(indptr), SCALE)
    _clean()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    _check_sparse(pool, fmt, 64, slots, indptr, q, out, lse, rows=[0, 2])


def test_fp8_scales_over_their_range():
    """Groups with scales from 2^-100 up to 2^9 in one row: undone exactly in bf16."""
    rng = np.random.default_rng(8)
    pool = ref.make_pool(rng, ref.FP8, 3, 64)
    pool[:, 64 * 640:] = rng.choice([27, 60, 100, 118, 120, 127, 134, 135, 136], pool[:, 64 * 640:].shape)
    slots = rng.permutation(192).astype(np.int32)
    indptr = np.array([0, 192], np.int32)
    qt, q = _bf16(1e-5 * rng.standard_normal((1, 16, 576)))
    out, lse = B.idx_latent_attention(qt, _dev(pool), 64, ref.FP8, _dev(slots), _dev(indptr), SCALE)
    _clean()
    _check_sparse(pool, ref.FP8, 64, slots, indptr, q, out, lse)


def _paged_case(rng, fmt, ctx, page, spare=2):
    need = [max(0, -(-c // page)) for c in ctx]
    pages = sum(need) + spare
    pool = ref.make_pool(rng, fmt, pages, page)
    perm = rng.permutation(pages).astype(np.int32)
    bt = np.full((len(ctx), max(need + [1]) + 1), 2 ** 30, np.int32)
    at, slots = 0, []
    for b, c in enumerate(ctx):
        bt[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        pos = np.arange(max(c, 0))
        slots.append(bt[b, pos // page].astype(np.int64) * page + pos % page)
    ref.poison(pool, fmt, page, np.concatenate(slots))
    return pool, bt, slots


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("ctx,next_n,H,page", [([1], 1, 16, 64), ([1, 300, 2], 3, 8, 64), ([64, 65, 63, 0], 1, 32, 16),
                                               ([129, 4096], 2, 64, 48), ([1000] * 3, 4, 128, 64),
                                               ([9000], 1, 16, 64)])
def test_paged(fmt, ctx, next_n, H, page):
    rng = np.random.default_rng(sum(ctx) + H)
    pool, bt, slots = _paged_case(rng, fmt, ctx, page)
    qt, q = _bf16(rng.standard_normal((len(ctx) * next_n, H, 576)))
    out, lse = B.idx_paged_latent_attention(qt, _dev(pool), page, fmt, _dev(bt), _dev(np.array(ctx, np.int32)),
                                            next_n, SCALE, max(ctx))
    _clean()
    out, lse = _np(out), _np(lse)
    for b, c in enumerate(ctx):
        tok = ref.read_tokens(pool, fmt, page, slots[b])
        for j in range(next_n):
            t = tok[:max(0, c - next_n + j + 1)]
            ref.check(out[b * next_n + j], lse[b * next_n + j], ref.attend(q[b * next_n + j], t, t[:, :512], SCALE))


@pytest.mark.parametrize("fmt", FMTS)
def test_paged_lengths_per_row_and_clamped(fmt):
    """One length a row, lengths outside [0, max_model_len] and a page outside the pool."""
    rng = np.random.default_rng(11)
    pool, bt, slots = _paged_case(rng, fmt, [200, 130], 64)
    qt, q = _bf16(rng.standard_normal((4, 16, 576)))
    per_row = np.array([-3, 77, 500, 130], np.int32)
    bt[1, 1] = -1
    out, lse = B.idx_paged_latent_attention(qt, _dev(pool), 64, fmt, _dev(bt), _dev(per_row), 2, SCALE, 130,
                                            ctx_per_row=True)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_PAGE
    out, lse = _np(out), _np(lse)
    for r, n in enumerate([0, 77, 130, 130]):
        pos = np.arange(n)
        s = slots[r // 2][:n] if r < 2 else slots[1][:n][(pos < 64) | (pos >= 128)]
        tok = ref.read_tokens(pool, fmt, 64, s)
        ref.check(out[r], lse[r], ref.attend(q[r], tok, tok[:, :512], SCALE))


@pytest.mark.parametrize("fmt", FMTS)
def test_same_bits_again_other_stream_and_graph(fmt):
    rng = np.random.default_rng(12)
    pool, slots, indptr, qt, q = _sparse_case(rng, fmt, [2000, 130, 0, 64] * 3, 64, 64)
    args = (qt, _dev(pool), 64, fmt, _dev(slots), _dev(indptr), SCALE)
    first, lse = B.idx_latent_attention(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = B.prepare_latent_attention(*args)
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(call.keep[4], first) and torch.equal(call.keep[5], lse)
    for _ in range(3):  # outputs and scratch made for the stream they are written on
        other, _ = B.idx_latent_attention(*args, stream=side)
        side.synchronize()
        assert torch.equal(other, first)
    call.keep[4].zero_()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        g.replay()
    _clean()
    assert torch.equal(call.keep[4], first)
    _check_sparse(pool, fmt, 64, slots, indptr, q, first, lse)


# ------------------------------------------------------------- expanded attention


def _prefill_case(rng, lq, lk, H, tail=5):
    nq, nk = sum(lq), sum(lk)
    cq = np.concatenate([[0], np.cumsum(lq)]).astype(np.int32)
    ck = np.concatenate([[0], np.cumsum(lk)]).astype(np.int32)
    qt, q = _bf16(rng.standard_normal((nq, H, 192)))
    kv = rng.standard_normal((nk + tail, H, 256))
    lat = rng.standard_normal((nk + tail, 576))
    kv[nk:], lat[nk:] = np.nan, np.nan  # past the last sequence
    kvt, kv = _bf16(kv)
    latt, lat = _bf16(lat)
    return cq, ck, qt, q, kvt, kv, latt, lat


def _check_prefill(cq, ck, q, kv, rope, out, lse, causal, seqs=None):
    out, lse = _np(out), _np(lse)
    for b in range(len(cq) - 1) if seqs is None else seqs:
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        seen = np.arange(nk)[None] <= (np.arange(nq) + nk - nq)[:, None] if causal else None
        for h in range(q.shape[1]):
            k = np.concatenate([kv[ck[b]:ck[b + 1], h, :128], rope[ck[b]:ck[b + 1]]], 1)
            got = out[cq[b]:cq[b + 1], h]
            ref.check(got, lse[cq[b]:cq[b + 1], h],
                      ref.attend(q[cq[b]:cq[b + 1], h], k, kv[ck[b]:ck[b + 1], h, 128:], SCALE, seen))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,H", [([1], [1], 1), ([1, 1], [700, 1], 3), ([0, 5, 0], [3, 5, 0], 2),
                                     ([127, 128, 129], [127, 128, 129], 2), ([64, 65, 257], [64, 400, 300], 3),
                                     ([300], [200], 2), ([5, 130], [0, 130], 1), ([513], [1300], 2),
                                     ([1] * 70, [33] * 70, 2)])
def test_prefill(lq, lk, H, causal):
    rng = np.random.default_rng(sum(lq) + sum(lk))
    cq, ck, qt, q, kvt, kv, latt, lat = _prefill_case(rng, lq, lk, H)
    out, lse = B.idx_latent_prefill(qt, kvt[..., :128], latt[:, 512:], kvt[..., 128:], _dev(cq), _dev(ck), SCALE,
                                    causal=causal)
    _clean()
    _check_prefill(cq, ck, q, kv, lat[:, 512:], out, lse, causal)


def test_prefill_strides_unlisted_rows_and_other_sequences():
    """Strided q and out; query rows past the last sequence stay untouched; a
    sequence of NaN next to others does not reach them."""
    rng = np.random.default_rng(21)
    lq, lk, H = [70, 40, 90], [100, 150, 90], 3
    cq, ck, _, _, kvt, kv, latt, lat = _prefill_case(rng, lq, lk, H)
    kvt[100:250] = float("nan")
    latt[100:250] = float("nan")
    big, q = _bf16(rng.standard_normal((206, 5, 200)))
    o = torch.full((206, 5, 136), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((206, 4), 3.0, device="cuda")
    B.idx_latent_prefill(big[:, 1:4, :192], kvt[..., :128], latt[:, 512:], kvt[..., 128:], _dev(cq), _dev(ck), SCALE,
                         out=o[:, 2:5, :128], lse=lse[:, :3])
    _clean()
    _check_prefill(cq, ck, q[:, 1:4, :192], kv, lat[:, 512:], o[:, 2:5, :128], lse[:, :3], True, seqs=[0, 2])
    assert torch.isnan(o[70:110, 2:5, :128]).all()
    assert (o[200:] == 3).all() and (o[:, :2] == 3).all() and (o[..., 128:] == 3).all()
    assert (lse[200:] == 3).all() and (lse[:, 3] == 3).all()


def test_prefill_peaked_and_graph():
    rng = np.random.default_rng(22)
    cq, ck, qt, q, kvt, kv, latt, lat = _prefill_case(rng, [200, 333], [600, 333], 2)
    qt, q = _bf16(20 * q)
    call = B.prepare_latent_prefill(qt, kvt[..., :128], latt[:, 512:], kvt[..., 128:], _dev(cq), _dev(ck), SCALE)
    call()
    _clean()
    first = call.keep[6].clone()
    _check_prefill(cq, ck, q, kv, lat[:, 512:], first, call.keep[7], True)
    call.keep[6].zero_()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call()
    g.replay()
    _clean()
    assert torch.equal(call.keep[6], first)


# --------------------------------------------------- sizes where the lists end


@pytest.mark.parametrize("fmt", FMTS)
def test_sparse_more_rows_than_threads(fmt):
    """The share scan's threads take several rows each; one row is cut."""
    rng = np.random.default_rng(41)
    lens = np.concatenate([rng.integers(0, 9, 1100), [700], rng.integers(0, 9, 300)])
    pool, slots, indptr, qt, q = _sparse_case(rng, fmt, lens, 8, 64)
    out, lse = B.idx_latent_attention(qt, _dev(pool), 64, fmt, _dev(slots), _dev(indptr), SCALE)
    _clean()
    _check_sparse(pool, fmt, 64, slots, indptr, q, out, lse, rows=list(range(0, 1401, 37)) + [1100])


def test_sparse_bounds_past_the_slots():
    """Row bounds outside the listed slots are clamped to them."""
    rng = np.random.default_rng(42)
    pool, slots, indptr, qt, q = _sparse_case(rng, ref.FP8, [100, 90, 60], 16, 64)
    wrong = np.array([-5, 100, 10 ** 9, 2 ** 31 - 1], np.int32)
    out, lse = B.idx_latent_attention(qt, _dev(pool), 64, ref.FP8, _dev(slots), _dev(wrong), SCALE)
    _clean()
    _check_sparse(pool, ref.FP8, 64, slots, np.array([0, 100, 250, 250]), q, out, lse)


@pytest.mark.parametrize("fmt", FMTS)
def test_sparse_heads_before_rows(fmt):
    """Queries and outputs laid out [H, R, ..]: the head stride is the larger."""
    rng = np.random.default_rng(43)
    pool, slots, indptr, _, _ = _sparse_case(rng, fmt, [300, 5, 64], 20, 64)
    t, q = _bf16(rng.standard_normal((20, 3, 576)))
    o = torch.empty(20, 3, 512, dtype=torch.bfloat16, device="cuda")
    out, lse = B.idx_latent_attention(t.transpose(0, 1), _dev(pool), 64, fmt, _dev(slots), _dev(indptr), SCALE,
                                      out=o.transpose(0, 1))
    _clean()
    _check_sparse(pool, fmt, 64, slots, indptr, q.transpose(1, 0, 2), out, lse)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("next_n,H", [(3, 24), (2, 40), (5, 16), (4, 1)])
def test_paged_rows_sharing_columns(fmt, next_n, H):
    """Groups of columns that hold some of a sequence's rows, the last one fewer."""
    rng = np.random.default_rng(next_n * H)
    ctx, page = [next_n - 1, 130, 1100], 64
    pool, bt, slots = _paged_case(rng, fmt, ctx, page)
    qt, q = _bf16(rng.standard_normal((len(ctx) * next_n, H, 576)))
    out, lse = B.idx_paged_latent_attention(qt, _dev(pool), page, fmt, _dev(bt), _dev(np.array(ctx, np.int32)),
                                            next_n, SCALE, max(ctx))
    _clean()
    out, lse = _np(out), _np(lse)
    for b, c in enumerate(ctx):
        tok = ref.read_tokens(pool, fmt, page, slots[b])
        for j in range(next_n):
            t = tok[:max(0, c - next_n + j + 1)]
            ref.check(out[b * next_n + j], lse[b * next_n + j], ref.attend(q[b * next_n + j], t, t[:, :512], SCALE))


@pytest.mark.parametrize("fmt", FMTS)
def test_cache_beyond_four_gigabytes(fmt):
    """Store, read-back and attention at byte offsets past 2^32."""
    rng = np.random.default_rng(44)
    page, stride = 64, ref.page_stride(fmt, 64)
    pages = (2 ** 32 + 2 ** 30) // stride
    pool = torch.empty(pages, stride, dtype=torch.uint8, device="cuda")
    slots = np.concatenate([np.arange(100), pages * page - 200 + np.arange(200)]).astype(np.int64)
    t, x = _bf16(rng.standard_normal((300, 576)))
    B.idx_latent_store(t, None, None, None, 0.0, pool, page, _dev(slots), fmt)
    bt = np.array([[0, 1, pages - 4, pages - 3, pages - 2, pages - 1]], np.int32)
    back = torch.empty(6 * page, 576, dtype=torch.bfloat16, device="cuda")
    B.idx_latent_gather(pool, page, fmt, _dev(bt), _dev(np.array([0, 6 * page], np.int32)), back)
    _clean()
    got = _np(back)
    at = np.concatenate([np.arange(100), 6 * page - 200 + np.arange(200)])
    tol = 0 if fmt == ref.BF16 else 2.0 ** -4 * np.abs(x) + 2.0 ** -10
    assert (np.abs(got[at] - x) <= tol).all()
    qt, q = _bf16(rng.standard_normal((1, 16, 576)))
    out, lse = B.idx_latent_attention(qt, pool, page, fmt, _dev(slots.astype(np.int32)),
                                      _dev(np.array([0, 300], np.int32)), SCALE)
    _clean()
    ref.check(_np(out)[0], _np(lse)[0], ref.attend(q[0], got[at], got[at][:, :512], SCALE))


@pytest.mark.parametrize("count", [200, 900])
def test_prefill_many_sequences(count):
    """More sequences than the kernel keeps bounds for, and than it has threads."""
    rng = np.random.default_rng(count)
    lq = rng.integers(0, 4, count).tolist()
    lk = [a + int(b) for a, b in zip(lq, rng.integers(0, 3, count))]
    lq[count // 2], lk[count // 2] = 300, 700
    cq, ck, qt, q, kvt, kv, latt, lat = _prefill_case(rng, lq, lk, 2)
    out, lse = B.idx_latent_prefill(qt, kvt[..., :128], latt[:, 512:], kvt[..., 128:], _dev(cq), _dev(ck), SCALE)
    _clean()
    _check_prefill(cq, ck, q, kv, lat[:, 512:], out, lse, True)


def test_prefill_without_keys_and_one_long_row():
    z = torch.zeros(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(5, 2, 192, dtype=torch.bfloat16, device="cuda")
    cu = lambda *a: _dev(np.array(a, np.int32))  # noqa: E731
    out, lse = B.idx_latent_prefill(q, z, z[:, 0, :64], z, cu(0, 5), cu(0, 0), SCALE)
    _clean()
    assert (out == 0).all() and (lse == -float("inf")).all()
    # one query on many keys: cut over the whole GPU
    rng = np.random.default_rng(45)
    cq, ck, qt, qn, kvt, kv, latt, lat = _prefill_case(rng, [1], [40000], 1)
    out, lse = B.idx_latent_prefill(qt, kvt[..., :128], latt[:, 512:], kvt[..., 128:], _dev(cq), _dev(ck), SCALE)
    _clean()
    _check_prefill(cq, ck, qn, kv, lat[:, 512:], out, lse, True)


def test_nothing_to_do():
    bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = torch.zeros(2, 64 * 648, dtype=torch.uint8, device="cuda")
    B.idx_latent_store(bf(0, 576), None, None, None, 0.0, pool, 64, torch.zeros(0, dtype=torch.int64, device="cuda"), 1)
    B.idx_latent_gather(pool, 64, 1, i32(1, 2), i32(2), bf(0, 576))
    out, lse = B.idx_latent_attention(bf(0, 4, 576), pool, 64, 1, i32(0), i32(1), SCALE)
    assert out.shape == (0, 4, 512) and lse.shape == (0, 4)
    out, lse = B.idx_latent_prefill(bf(0, 4, 192), bf(3, 4, 128), bf(3, 64), bf(3, 4, 128), i32(2), i32(2), SCALE)
    assert out.shape == (0, 4, 128)
    _clean()


@pytest.mark.parametrize("H,rows,mix", [(16, 700, (0, 3)), (16, 160, (0, 200)), (64, 153, (0, 130)), (64, 40, (60, 70)),
                                        (128, 90, (1, 500)), (24, 19, (300, 2000)), (64, 9, (1000, 1100)),
                                        (3, 2, (5000, 9000))])
def test_sparse_random_lists(H, rows, mix):
    """Shares that begin and end anywhere in a list of rows, within what a row
    is charged too; the bits do not change from call to call."""
    rng = np.random.default_rng(rows + H)
    lens = rng.integers(mix[0], mix[1] + 1, rows)
    pool, slots, indptr, q, qv = _sparse_case(rng, ref.FP8, lens, H, 64)
    args = _dev(pool), 64, ref.FP8, _dev(slots), _dev(indptr), SCALE
    out, lse = B.idx_latent_attention(q, *args)
    _clean()
    some = rng.choice(rows, min(rows, 12), replace=False)
    _check_sparse(pool, ref.FP8, 64, slots, indptr, qv, out, lse, rows=some)
    again, lse2 = B.idx_latent_attention(q, *args)
    _clean()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H,seqs,longest", [(1, 40, 300), (3, 12, 700), (5, 7, 1500), (16, 3, 900), (2, 150, 140)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_random_packs(H, seqs, longest, causal):
    """Blocks of one and two query tiles in every order, cut by shares and not,
    with contexts before some of the prompts and rows without keys."""
    rng = np.random.default_rng(H * 1000 + seqs)
    lq = rng.integers(0, longest, seqs)
    lk = np.maximum(0, lq + rng.integers(-60, 300, seqs))
    cq, ck, qt, q, kvt, kv, latt, lat = _prefill_case(rng, lq, lk, H)
    call = lambda: B.idx_latent_prefill(qt, kvt[..., :128], latt[:, 512:], kvt[..., 128:], _dev(cq), _dev(ck),  # noqa: E731
                                        SCALE, causal=causal)
    out, lse = call()
    _clean()
    picked = sorted(rng.choice(seqs, min(seqs, 6), replace=False))
    _check_prefill(cq, ck, q, kv, lat[:, 512:], out, lse, causal, seqs=picked)
    again, lse2 = call()
    _clean()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
