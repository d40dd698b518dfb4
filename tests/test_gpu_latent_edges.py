"""GPU checks of the latent calls where inputs are at an edge: tokens that are
not finite, values at the ends of the types' range, layouts of one row or one
head, bounds past their tensors, packs and scratch at their limits."""
import numpy as np
import pytest
import torch

import latent_ref as ref
from sparse_attention_indexer_mxfp4_gb300 import LatentLayer
from sparse_attention_indexer_mxfp4_gb300 import _binding as B
from test_gpu_latent import (SCALE, _bf16, _check_prefill, _check_sparse, _clean, _dev, _np, _paged_case,
                             _prefill_case, _sparse_case)
from test_latent_calls_host import CALLS
from test_latent_edges_host import Elsewhere

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


# ------------------------------------------- tokens that a row is not to see


def _token_put(pool, fmt, page, slot, what):
    """Makes one cached token NaN, or infinite in latent 7."""
    line, o = pool[slot // page], slot % page
    if fmt == ref.BF16:
        word = {"nan": 0x7fc0, "inf": 0x7f80, "-inf": 0xff80}[what]
        line[o * 1152 + 14:o * 1152 + 16] = word & 255, word >> 8
    elif what == "nan":
        line[page * 640 + o * 8 + 3] = 255  # latents 192 .. 255
    else:
        line[o * 512:o * 512 + 64] = 0
        line[o * 512 + 7] = {"inf": 0x7e, "-inf": 0xfe}[what]  # 448 * 2^127 is past bf16
        line[page * 640 + o * 8] = 254


def _attend_ieee(q, tok, seen):
    """The formula with IEEE's rules: a NaN score or an infinite one at the top
    makes the row NaN; a weight of zero times an infinity is NaN."""
    t = tok[:seen].copy()
    t[np.isinf(t) | (np.abs(t) > 3.39e38)] *= np.inf
    with np.errstate(invalid="ignore"):
        s = q @ t.T
    every = np.isnan(s).any(1) | (s == np.inf).any(1)
    lost = ~np.isfinite(t[:, :512]).all(0)  # latents
    keep = np.isfinite(t).all(1)
    return every, lost, ref.attend(q, t[keep], t[keep][:, :512], SCALE)


def _check_hidden(out, lse, q, tok, ends):
    for r, end in enumerate(ends):
        every, lost, want = _attend_ieee(q[r], tok, end)
        assert np.isnan(out[r][every]).all() and np.isnan(lse[r][every]).all()
        o, l, pv, mag = (x[~every] for x in want)
        assert np.isnan(out[r][~every][:, lost]).all()
        ref.check(out[r][~every][:, ~lost], lse[r][~every], (o[:, ~lost], l, pv[:, ~lost], mag))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("ctx,next_n,H", [(130, 2, 16), (65, 2, 64), (66, 3, 8), (3, 3, 16), (64, 4, 1), (128, 2, 128),
                                          (2000, 2, 24), (2, 2, 40)])
def test_paged_tokens_past_a_rows_end(fmt, what, ctx, next_n, H):
    """The newest tokens of a sequence are not finite: rows that end before them are as if they were not there."""
    rng = np.random.default_rng(ctx + H)
    pool, bt, slots = _paged_case(rng, fmt, [ctx, 70], 64)
    for k in {0, next_n - 2}:  # the last token, and the oldest that some row does not see
        _token_put(pool, fmt, 64, slots[0][ctx - 1 - k], what)
    qt, q = _bf16(rng.standard_normal((2 * next_n, H, 576)))
    out, lse = B.idx_paged_latent_attention(qt, _dev(pool), 64, fmt, _dev(bt), _dev(np.array([ctx, 70], np.int32)),
                                            next_n, SCALE, max(ctx, 70))
    _clean()
    out, lse = _np(out), _np(lse)
    for b, c in enumerate([ctx, 70]):
        rows = slice(b * next_n, (b + 1) * next_n)
        tok = ref.read_tokens(pool, fmt, 64, slots[b])
        _check_hidden(out[rows], lse[rows], q[rows], tok, [max(0, c - next_n + j + 1) for j in range(next_n)])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("per_row,bad,H", [([0, 130, 64, 1], [64], 16), ([0, 130, 64, 1], [0], 64), ([0, 1], [0], 16),
                                           ([700, 3000, 2001], [700, 2000, 2999], 16), ([-4, 5000], [1, 3000], 128),
                                           ([64, 64, 200], [100, 150], 8)])
def test_paged_lengths_per_row_hide_tokens(fmt, what, per_row, bad, H):
    """Lengths given row by row, far apart: a row of none stays zeros, a short one its own."""
    rng = np.random.default_rng(sum(per_row) + H)
    longest = max(per_row)
    pool, bt, slots = _paged_case(rng, fmt, [longest], 64)
    for t in bad:
        _token_put(pool, fmt, 64, slots[0][t], what)
    qt, q = _bf16(rng.standard_normal((len(per_row), H, 576)))
    out, lse = B.idx_paged_latent_attention(qt, _dev(pool), 64, fmt, _dev(bt), _dev(np.array(per_row, np.int32)),
                                            len(per_row), SCALE, longest, ctx_per_row=True)
    _clean()
    _check_hidden(_np(out), _np(lse), q, ref.read_tokens(pool, fmt, 64, slots[0]), [max(0, n) for n in per_row])


def test_paged_hidden_nan_code():
    """A NaN code past a row's end, among the largest finite ones."""
    rng = np.random.default_rng(4)
    pool, bt, slots = _paged_case(rng, ref.FP8, [100], 64)
    for s in slots[0]:
        pool[s // 64, (s % 64) * 512:][:512:5] = rng.choice([0x7e, 0xfe, 0x77, 0xf7, 0x6f], 103)
    s = slots[0][99]
    pool[s // 64, (s % 64) * 512 + 9] = 0xff
    qt, q = _bf16(0.01 * rng.standard_normal((2, 16, 576)))
    out, lse = B.idx_paged_latent_attention(qt, _dev(pool), 64, ref.FP8, _dev(bt), _dev(np.array([100], np.int32)), 2,
                                            SCALE, 100)
    _clean()
    _check_hidden(_np(out), _np(lse), q, ref.read_tokens(pool, ref.FP8, 64, slots[0]), [99, 100])


# ------------------------------------------------------------------- devices


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_of_a_device_that_is_not_current(name):
    """Refused before a pointer is taken: the tensors have no storage."""
    call, prepare, good = CALLS[name]
    args = [Elsewhere(x.shape, x.dtype, "cuda:1") if torch.is_tensor(x) else x for x in good()]
    for f in (call, prepare):
        with pytest.raises(ValueError, match="current device is cuda:0"):
            f(*args)


# ------------------------------------------------------ bounds past the tensors


@pytest.mark.parametrize("fmt", FMTS)
def test_gather_tells_of_rows_that_do_not_fit(fmt):
    rng = np.random.default_rng(2)
    pool = ref.make_pool(rng, fmt, 3, 64)
    out = torch.full((100, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    B.idx_latent_gather(_dev(pool), 64, fmt, _dev(np.array([[2, 1]], np.int32)), _dev(np.array([0, 101], np.int32)), out)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_BOUNDS
    want = ref.read_tokens(pool, fmt, 64, np.concatenate([128 + np.arange(64), 64 + np.arange(36)]))
    assert np.array_equal(_np(out), want)


@pytest.mark.parametrize("cu_q,cu_k", [([0, 5, 11], [0, 9, 20]), ([0, 5, 10], [0, 9, 21]), ([0, 5, 10], [-1, 9, 20]),
                                       ([0, 11, 10], [0, 9, 20])])
def test_prefill_tells_of_bounds_past_its_tensors(cu_q, cu_k):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    B.idx_latent_prefill(z(10, 2, 192), z(20, 2, 128), z(20, 64), z(20, 2, 128), _dev(np.array(cu_q, np.int32)),
                         _dev(np.array(cu_k, np.int32)), SCALE)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_BOUNDS


def test_layer_tells_of_too_few_tokens():
    """A prefill told of fewer cached tokens than its bounds have is not silently cut."""
    rng = np.random.default_rng(5)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s)).bfloat16().cuda()  # noqa: E731
    layer = LatentLayer(t(2, 128, 512), t(2, 128, 512), torch.ones(512, device="cuda"),
                        torch.ones(64, 64, device="cuda"), 4, 64)
    layer.store(t(60, 576), torch.arange(60, dtype=torch.int32, device="cuda"), torch.arange(60, device="cuda"))
    cu = torch.tensor([0, 60], dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    layer.prefill(t(60, 2, 192), cu, table, cu, 60)
    _clean()
    layer.prefill(t(60, 2, 192), cu, table, cu, 59)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_BOUNDS


def test_list_that_descends():
    """Rows named again by bounds that descend are computed while the list can be counted; a list that cannot is left
    alone, told of, and harms no later call."""
    rng = np.random.default_rng(43)
    pool, slots, _, qt, q = _sparse_case(rng, ref.FP8, [700], 16, 64)
    qt, q = _bf16(rng.standard_normal((5, 16, 576)))
    falls = np.array([0, 700, 0, 300, 100, 650], np.int32)
    args = _dev(pool), 64, ref.FP8, _dev(slots)
    out, lse = B.idx_latent_attention(qt, *args, _dev(falls), SCALE)
    _clean()
    _check_sparse(pool, ref.FP8, 64, slots, falls, q, out, lse)
    rows, n = 1 << 18, 1 << 20  # half of the rows name all of a million slots
    far = torch.zeros(rows + 1, dtype=torch.int32, device="cuda")
    far[1::2] = n
    many = torch.zeros(n, dtype=torch.int32, device="cuda")
    B.idx_latent_attention(torch.zeros(rows, 1, 576, dtype=torch.bfloat16, device="cuda"), *args[:3], many, far, SCALE)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_BOUNDS
    again, _ = B.idx_latent_attention(qt, *args, _dev(falls), SCALE)
    _clean()
    assert torch.equal(again, out)


# --------------------------------------------------------- long lists of work


def test_prefill_pack_of_many_sequences_and_heads():
    """20000 sequences of 70 heads: every block times all keys is past 32 bits, the list is not."""
    B_, H, lk = 20000, 70, 10
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q, kv, lat = r(B_, H, 192), r(B_ * lk, H, 256), r(B_ * lk, 64)
    cu_q = torch.arange(B_ + 1, dtype=torch.int32, device="cuda")
    cu_k = cu_q * lk
    out, lse = B.idx_latent_prefill(q, kv[..., :128], lat, kv[..., 128:], cu_q, cu_k, SCALE)
    _clean()
    for b in [0, 1, 383, 384, 9999, 12345, 19999]:
        k = slice(b * lk, b * lk + lk)
        _check_prefill(np.array([0, 1]), np.array([0, lk]), _np(q[b:b + 1]), _np(kv[k]), _np(lat[k]), out[b:b + 1],
                       lse[b:b + 1], True)
    # each of the equal sequences is computed: none has kept what was in memory
    assert torch.isfinite(out).all() and (out.abs().amax(-1) > 0).all()


def test_prefill_list_that_cannot_be_counted():
    """Bounds that descend name the same tokens again and again: told of, and no later call is harmed."""
    n, H, seqs = 1 << 16, 64, 1 << 15
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, k, rope = z(n, H, 192), z(n, H, 128), z(n, 64)
    far = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    far[1::2] = n
    B.idx_latent_prefill(q, k, rope, k, far, far, SCALE, causal=False)
    torch.cuda.synchronize()
    assert B.idx_get_device_status() == B.DEV_BAD_BOUNDS
    del q, k
    rng = np.random.default_rng(9)
    cq, ck, qt, qv, kvt, kv, latt, lat = _prefill_case(rng, [300], [900], 2)
    out, lse = B.idx_latent_prefill(qt, kvt[..., :128], latt[:, 512:], kvt[..., 128:], _dev(cq), _dev(ck), SCALE)
    _clean()
    _check_prefill(cq, ck, qv, kv, lat[:, 512:], out, lse, True)


# --------------------------------------------------- values at the types' ends


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-6, 4.0])
def test_store_norm_of_large_and_small_tokens(fmt, eps):
    """Squares past 32 bits' range on either side: the norm is the formula's."""
    rng = np.random.default_rng(6)
    size = np.array([3e38, 1e30, 1e19, 1e17, 1.0, 1e-12, 1e-15, 1e-18, 1e-25, 1e-36])
    x = np.clip(rng.standard_normal((len(size), 576)), -1, 1) * size[:, None]
    x[:, 512:] = 0
    t, v = _bf16(x)
    w = (1 + 0.1 * rng.standard_normal(512)).astype(np.float32)
    page = 16
    pool = torch.zeros(1, ref.page_stride(fmt, page), dtype=torch.uint8, device="cuda")
    slots = np.arange(len(size))
    B.idx_latent_store(t, None, None, _dev(w), eps, pool, page, _dev(slots), fmt)
    _clean()
    y = v[:, :512] / np.sqrt((v[:, :512] ** 2).mean(1, keepdims=True) + eps) * w
    got = ref.read_tokens(pool.cpu().numpy(), fmt, page, slots)[:, :512]
    if fmt == ref.BF16:
        # half a step, subnormal ones among them, and a few units of the 32-bit norm
        assert (np.abs(got - y) <= (ref.HALF_BF16 + 2.0 ** -20) * np.abs(y) + 2.0 ** -133).all()
    else:
        amax = np.repeat(np.abs(y).reshape(-1, 8, 64).max(-1), 64, 1).reshape(y.shape)
        # the group's step is at most amax / 224, or the least scale's
        step = np.maximum(amax / 224, 2.0 ** -127)
        assert (np.abs(got - y) <= (2.0 ** -4 + 1e-5) * np.abs(y) + (2.0 ** -10 + 1e-5) * step).all()


# ------------------------------------------------- layouts of one row, one head


def _odd(t, *dims):
    """The same tensor with strides of no meaning where it has one element."""
    strides = list(t.stride())
    for d in dims:
        assert t.shape[d] == 1
        strides[d] = 1
    return t.as_strided(t.shape, strides)


def test_strides_over_one_element_are_free():
    rng = np.random.default_rng(8)
    pool, slots, indptr, qt, q = _sparse_case(rng, ref.FP8, [70], 1, 128)
    dev = _dev(pool)
    one = _odd(dev[:1], 0)
    o, l = torch.empty(1, 1, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 1, device="cuda")
    out, lse = B.idx_latent_attention(_odd(qt, 0, 1), dev, 128, ref.FP8, _dev(slots), _dev(indptr), SCALE,
                                      out=_odd(o, 0, 1), lse=_odd(l, 0))
    _clean()
    _check_sparse(pool, ref.FP8, 128, slots, indptr, q, out, lse)
    # one token stored into a pool of one page, and read back
    kv, x = _bf16(rng.standard_normal((1, 576)))
    cs = torch.ones(1, 64, device="cuda")
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.idx_latent_store(_odd(kv, 0), pos, _odd(cs, 0), None, 0.0, one, 128, _dev(np.array([5])), ref.FP8)
    back = torch.empty(1, 576, dtype=torch.bfloat16, device="cuda")
    B.idx_latent_gather(one, 128, ref.FP8, _dev(np.zeros((1, 1), np.int32)), _dev(np.array([0, 1], np.int32)),
                        _odd(back, 0), seq_starts=_dev(np.array([5], np.int32)))
    _clean()
    assert (np.abs(_np(back)[:, :512] - x[:, :512]) <= 2.0 ** -4 * np.abs(x[:, :512]) + 2.0 ** -10).all()
    # one query on one key
    cq, ck, qt, q, kvt, kv, latt, lat = _prefill_case(rng, [1], [1], 1, tail=0)
    o = torch.empty(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    out, lse = B.idx_latent_prefill(_odd(qt, 0, 1), _odd(kvt[..., :128], 0, 1), _odd(latt[:, 512:], 0),
                                    _odd(kvt[..., 128:], 0, 1), _dev(cq), _dev(ck), SCALE, out=_odd(o, 0, 1))
    _clean()
    _check_prefill(cq, ck, q, kv, lat[:, 512:], out, lse, True)


# ----------------------------------------------------- launches that are counted


def test_launches_of_prepared_calls():
    """The joining kernel is counted where rows are cut, and nothing where nothing is to do."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = torch.zeros(2, 64 * 648, dtype=torch.uint8, device="cuda")
    slots = lambda R, n: B.prepare_latent_attention(bf(R, 4, 576), pool, 64, 1, i32(n), i32(R + 1), SCALE).kernels  # noqa: E731
    assert [slots(0, 0), slots(3, 256), slots(3, 257)] == [0, 1, 2]
    for next_n in (1, sms // 2, sms // 2 + 1, sms):  # 64 heads: a group of columns a row
        call = B.prepare_paged_latent_attention(bf(next_n, 64, 576), pool, 64, 1, i32(1, 20), i32(1), next_n, SCALE,
                                                1000)
        assert call.kernels == (2 if 2 * next_n <= sms else 1), next_n
        call()
    _clean()
    pre = lambda q, k, b: B.prepare_latent_prefill(bf(q, 2, 192), bf(k, 2, 128), bf(k, 64), bf(k, 2, 128), i32(b + 1),  # noqa: E731
                                                   i32(b + 1), SCALE).kernels
    assert [pre(0, 9, 1), pre(4, 512, 1), pre(4, 513, 1), pre(4, 513, 0)] == [0, 1, 2, 0]
    out = lambda n, b: B.prepare_latent_gather(pool, 64, 1, i32(max(b, 1), 2), i32(b + 1), bf(n, 576)).kernels  # noqa: E731
    assert [out(0, 1), out(5, 0), out(5, 1)] == [0, 0, 1]
    put = lambda n: B.prepare_latent_store(bf(n, 576), None, None, None, 0.0, pool, 64, i32(n).long(), 1).kernels  # noqa: E731
    assert [put(0), put(3)] == [0, 1]


# ------------------------------- scratch and outputs that are given, rows that are cut


class _Scratch:
    """Scratch of exactly n bytes between guards, all of it NaN in 32 bits before the call."""

    def __init__(self, n):
        assert n > 0
        self.n, self.all = n, torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda")

    def __call__(self, less=0):
        return self.all[2048:2048 + self.n - less]

    def check(self):
        torch.cuda.synchronize()
        assert (self.all[:2048] == 255).all() and (self.all[2048 + self.n:] == 255).all()
        assert (self.all != 255).any()  # it was used


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,H", [([2000, 0, 700], 24), ([1, 5000], 128), ([300] * 200 + [1500], 8), ([2048] * 20, 64)])
def test_sparse_given_scratch_and_outputs_of_cut_rows(fmt, lens, H):
    rng = np.random.default_rng(sum(lens) + H)
    R = len(lens)
    pool, slots, indptr, _, _ = _sparse_case(rng, fmt, lens, H, 64)
    big, q = _bf16(rng.standard_normal((R, H + 6, 584)))
    o = torch.full((R, H + 6, 520), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((R, H + 4), 3.0, device="cuda")
    ws = _Scratch(B.latent_attention_workspace_size(R, H, len(slots)))
    args = big[:, 2:2 + H, :576], _dev(pool), 64, fmt, _dev(slots), _dev(indptr), SCALE
    with pytest.raises(B.IndexerError, match="WORKSPACE"):
        B.idx_latent_attention(*args, workspace=ws(16))
    got, gl = B.idx_latent_attention(*args, out=o[:, 3:3 + H, :512], lse=lse[:, :H], workspace=ws())
    _clean()
    ws.check()
    some = sorted({0, 1, R // 2, R - 1})
    _check_sparse(pool, fmt, 64, slots, indptr, q[:, 2:2 + H, :576], got, gl, rows=some)
    made, ml = B.idx_latent_attention(*args)
    assert torch.equal(made, got) and torch.equal(ml, gl)
    assert (o[:, :3] == 3).all() and (o[:, 3 + H:] == 3).all() and (o[..., 512:] == 3).all() and (lse[:, H:] == 3).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_paged_given_scratch_and_outputs_of_cut_rows(fmt):
    rng = np.random.default_rng(51)
    ctx, next_n, H = [1800, 3, 900], 2, 24
    pool, bt, slots = _paged_case(rng, fmt, ctx, 64)
    qt, q = _bf16(rng.standard_normal((6, H, 576)))
    o = torch.full((H + 1, 6, 520), 3.0, dtype=torch.bfloat16, device="cuda")  # heads before rows
    lse = torch.full((6, H + 4), 3.0, device="cuda")
    ws = _Scratch(B.latent_attention_workspace_size(6, H, 2000))
    out, gl = B.idx_paged_latent_attention(qt, _dev(pool), 64, fmt, _dev(bt), _dev(np.array(ctx, np.int32)), next_n, SCALE,
                                           1800, out=o[:H, :, :512].transpose(0, 1), lse=lse[:, :H], workspace=ws())
    _clean()
    ws.check()
    out, gl = _np(out), _np(gl)
    for b, c in enumerate(ctx):
        tok = ref.read_tokens(pool, fmt, 64, slots[b])
        for j in range(next_n):
            t = tok[:max(0, c - next_n + j + 1)]
            ref.check(out[2 * b + j], gl[2 * b + j], ref.attend(q[2 * b + j], t, t[:, :512], SCALE))
    assert (o[H:] == 3).all() and (o[..., 512:] == 3).all() and (lse[:, H:] == 3).all()


@pytest.mark.parametrize("lq,lk,H,causal", [([300, 70, 200], [1300, 150, 900], 3, True), ([16], [20000], 1, True),
                                            ([1, 40, 5], [3000, 90, 4000], 2, False), ([700, 1, 257], [700, 900, 257], 5, True)])
def test_prefill_given_scratch_and_outputs_of_cut_blocks(lq, lk, H, causal):
    """The middle sequence, where there is one, is NaN; rows past the last one and what lies beside a head stay as they were."""
    rng = np.random.default_rng(sum(lq) + H)
    cq, ck, _, _, kvt, kv, latt, lat = _prefill_case(rng, lq, lk, H)
    if len(lq) > 1:
        kvt[ck[1]:ck[2]] = float("nan")
        latt[ck[1]:ck[2]] = float("nan")
    n = sum(lq)
    big, q = _bf16(rng.standard_normal((n + 6, H + 2, 200)))
    o = torch.full((n + 6, H + 2, 136), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + 6, H + 1), 3.0, device="cuda")
    args = big[:, 1:1 + H, :192], kvt[..., :128], latt[:, 512:], kvt[..., 128:], _dev(cq), _dev(ck), SCALE
    ws = _Scratch(B.latent_prefill_workspace_size(n + 6, sum(lk) + 5, H))
    with pytest.raises(B.IndexerError, match="WORKSPACE"):
        B.idx_latent_prefill(*args, workspace=ws(16))
    got, gl = B.idx_latent_prefill(*args, causal=causal, out=o[:, 2:, :128], lse=lse[:, :H], workspace=ws())
    _clean()
    ws.check()
    seqs = [0, 2] if len(lq) > 1 else [0]
    _check_prefill(cq, ck, q[:, 1:1 + H, :192], kv, lat[:, 512:], got, gl, causal, seqs=seqs)
    if len(lq) > 1:
        assert torch.isnan(got[cq[1]:cq[2]]).all() and torch.isnan(gl[cq[1]:cq[2]]).all()
    assert (o[n:] == 3).all() and (o[:, :2] == 3).all() and (o[..., 128:] == 3).all()
    assert (lse[n:] == 3).all() and (lse[:, H] == 3).all()
    made, ml = B.idx_latent_prefill(*args, causal=causal)
    assert torch.equal(made[:n].nan_to_num(7), got[:n].nan_to_num(7)) and torch.equal(ml[:n].nan_to_num(7), gl[:n].nan_to_num(7))
