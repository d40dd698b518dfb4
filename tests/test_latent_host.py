"""CPU checks of the latent-attention calls: the 64-bit reference against
identities it must satisfy, and the refusals of the C entry points (every call
here fails its host checks, so no pointer is followed)."""
import ctypes

import numpy as np
import pytest
import torch

import latent_ref as ref
from sparse_attention_indexer_mxfp4_gb300 import _binding as B

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE = 0x10000


def test_absorbed_equals_expanded():
    """q_nope . (W_k c) = (W_k^T q_nope) . c, and P (c W_v) = (P c) W_v."""
    rng = np.random.default_rng(0)
    c, rope = rng.standard_normal((37, ref.L)), rng.standard_normal((37, ref.ROPE))
    wk, wv = rng.standard_normal((128, ref.L)) / 22, rng.standard_normal((128, ref.L)) / 22
    q = rng.standard_normal((5, 192))
    expanded = ref.attend(q, np.concatenate([c @ wk.T, rope], 1), c @ wv.T, 0.1)
    absorbed = ref.attend(np.concatenate([q[:, :128] @ wk, q[:, 128:]], 1),
                          np.concatenate([c, rope], 1), c, 0.1)
    assert np.allclose(expanded[1], absorbed[1])
    assert np.allclose(expanded[0], absorbed[0] @ wv.T)


def test_reference_rows_that_see_nothing():
    q, k = np.ones((2, 4)), np.ones((3, 4))
    out, lse, _, _ = ref.attend(q, k, np.ones((3, 2)), 1.0, np.array([[False] * 3, [True] * 3]))
    assert (out[0] == 0).all() and lse[0] == -np.inf and np.allclose(out[1], 1)
    out, lse, _, _ = ref.attend(q, k[:0], np.ones((0, 2)), 1.0)
    assert (out == 0).all() and (lse == -np.inf).all()


def test_reference_codes():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3_float(codes), want, equal_nan=True)


@pytest.mark.parametrize("fmt", [ref.BF16, ref.FP8])
def test_page_bytes(fmt):
    for page in (1, 3, 16, 64, 100):
        assert B.latent_page_bytes(page, fmt) == ref.page_stride(fmt, page)


def _caller(name, base, places):
    fn = getattr(B.lib(), name)

    def call(**kw):
        a = list(base)
        for k, v in kw.items():
            a[places[k]] = v
        return fn(*a)
    return call


def test_store_refusals():
    base = [FAKE, 576, FAKE, FAKE, 64, 100, FAKE, 1e-6, 4, 512, 64, 1, FAKE, 41472, 10, 64, FAKE, None]
    p = dict(kv=0, ld=1, pos=2, cs=3, ldcs=4, npos=5, w=6, eps=7, T=8, L=9, rope=10, fmt=11, pages=12,
             stride=13, np=14, P=15, slots=16)
    call = _caller("idx_latent_store", base, p)
    assert call(T=0) == 0
    for kw in (dict(T=-1), dict(ld=575), dict(kv=None), dict(slots=None), dict(pos=None), dict(eps=-1.0),
               dict(eps=float("nan")), dict(ldcs=63), dict(npos=-1), dict(fmt=2), dict(pages=None),
               dict(stride=41456), dict(P=0), dict(np=-1), dict(fmt=0)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(L=256), dict(rope=32), dict(kv=FAKE + 2), dict(ld=580), dict(w=FAKE + 4),
               dict(pages=FAKE + 8), dict(stride=41480), dict(np=2 ** 26)):
        assert call(**kw) == UNSUPPORTED, kw


def test_gather_refusals():
    base = [FAKE, 41472, 10, 64, 1, 512, 64, FAKE, 8, 8, FAKE, None, 2, 100, FAKE, 576, None]
    p = dict(pages=0, stride=1, np=2, P=3, fmt=4, L=5, rope=6, bt=7, bts=8, mb=9, cu=10, start=11, B=12,
             N=13, out=14, ldo=15)
    call = _caller("idx_latent_gather", base, p)
    assert call(N=0) == 0 and call(B=0) == 0
    for kw in (dict(N=-1), dict(B=-1), dict(bts=7), dict(ldo=575), dict(bt=None), dict(cu=None),
               dict(out=None), dict(fmt=-1), dict(stride=100), dict(pages=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(L=448), dict(out=FAKE + 8), dict(ldo=580), dict(pages=FAKE + 4)):
        assert call(**kw) == UNSUPPORTED, kw


def test_attention_refusals():
    base = [FAKE, 64 * 576, 576, FAKE, 41472, 10, 64, 1, FAKE, FAKE, 1000, 4, 64, 512, 64, 0.1, FAKE,
            64 * 512, 512, FAKE, 64, FAKE, 1 << 30, None]
    p = dict(q=0, qr=1, qh=2, pages=3, stride=4, np=5, P=6, fmt=7, slots=8, indptr=9, ns=10, R=11, H=12,
             L=13, rope=14, scale=15, out=16, outr=17, oh=18, lse=19, ldl=20, ws=21, wsb=22)
    call = _caller("idx_latent_attention", base, p)
    assert call(R=0) == 0
    for kw in (dict(R=-1), dict(H=0), dict(q=None), dict(out=None), dict(indptr=None), dict(slots=None),
               dict(ns=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(qh=500), dict(oh=500), dict(ldl=63), dict(fmt=3), dict(stride=41456), dict(qr=-8)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(H=129, ldl=129), dict(L=256), dict(rope=0), dict(q=FAKE + 2), dict(qr=64 * 576 + 4),
               dict(qh=580), dict(out=FAKE + 8), dict(outr=4), dict(pages=FAKE + 8)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(ws=None) == WORKSPACE and call(wsb=0) == WORKSPACE and call(ws=FAKE + 8) == WORKSPACE


def test_paged_attention_refusals():
    base = [FAKE, 64 * 576, 576, FAKE, 41472, 10, 64, 1, FAKE, 16, FAKE, 0, 2, 2, 1000, 64, 512, 64, 0.1,
            FAKE, 64 * 512, 512, None, 0, FAKE, 1 << 30, None]
    p = dict(q=0, bt=8, bts=9, ctx=10, B=12, next_n=13, mml=14, H=15, out=19, ws=24, wsb=25)
    call = _caller("idx_paged_latent_attention", base, p)
    assert call(B=0) == 0
    for kw in (dict(B=-1), dict(next_n=0), dict(mml=-1), dict(bts=15), dict(bt=None), dict(ctx=None),
               dict(B=2 ** 30, next_n=4), dict(q=None)):
        assert call(**kw) == INVALID, kw
    assert call(H=200) == UNSUPPORTED and call(wsb=0) == WORKSPACE


def test_prefill_refusals():
    base = [FAKE, 64 * 192, 192, FAKE, 64 * 256, 256, FAKE, 576, FAKE, 64 * 256, 256, FAKE, FAKE, 2, 100,
            1000, 64, 128, 64, 128, 0.1, 1, FAKE, 64 * 128, 128, FAKE, 64, FAKE, 1 << 30, None]
    p = dict(q=0, qr=1, qh=2, k=3, kr=4, kh=5, rope=6, ldr=7, v=8, vr=9, vh=10, cq=11, ck=12, B=13, Tq=14,
             Tk=15, H=16, dn=17, dr=18, dv=19, scale=20, out=22, outr=23, oh=24, lse=25, ldl=26, ws=27, wsb=28)
    call = _caller("idx_latent_prefill", base, p)
    assert call(B=0) == 0 and call(Tq=0) == 0
    for kw in (dict(B=-1), dict(Tq=-1), dict(Tk=-1), dict(H=0), dict(q=None), dict(k=None), dict(rope=None),
               dict(v=None), dict(cq=None), dict(ck=None), dict(out=None), dict(scale=-1.0), dict(qh=184),
               dict(kh=120), dict(ldr=56), dict(vh=120), dict(oh=120), dict(ldl=63), dict(qr=-8)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dn=64), dict(dr=32), dict(dv=64), dict(q=FAKE + 2), dict(kr=64 * 256 + 4), dict(ldr=572),
               dict(v=FAKE + 8), dict(H=65536, ldl=65536)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(ws=None) == WORKSPACE and call(wsb=0) == WORKSPACE and call(ws=FAKE + 8) == WORKSPACE


def test_binding_refusals():
    """Shapes and types are refused before the library is called."""
    bf = torch.bfloat16
    z = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d)  # noqa: E731
    pool, q = z(4, 41472, d=torch.uint8), z(3, 16, 576, d=bf)
    with pytest.raises(ValueError):
        B.prepare_latent_attention(q.float(), pool, 64, 1, z(5), z(4), 0.1)
    with pytest.raises(ValueError):
        B.prepare_latent_attention(q, pool, 64, 1, z(5), z(3), 0.1)
    with pytest.raises(ValueError):
        B.prepare_latent_attention(q[..., :512], pool, 64, 1, z(5), z(4), 0.1)
    with pytest.raises(ValueError):
        B.prepare_latent_attention(q, pool, 64, 1, z(5), z(4), 0.1, out=z(3, 16, 500, d=bf))
    with pytest.raises(ValueError):
        B.prepare_latent_attention(q, pool, 64, 1, z(5), z(4), 0.1, lse=z(3, 16))
    with pytest.raises(ValueError):
        B.prepare_paged_latent_attention(q, pool, 64, 1, z(3, 2), z(3), 2, 0.1, 100)
    with pytest.raises(ValueError):
        B.prepare_paged_latent_attention(q, pool, 64, 1, z(2, 2), z(3), 1, 0.1, 100)
    with pytest.raises(ValueError):
        B.prepare_latent_store(z(2, 576, d=bf), None, z(4, 64, d=torch.float32), None, 0.0, pool, 64,
                               z(2, d=torch.int64), 1)
    with pytest.raises(ValueError):
        B.prepare_latent_store(z(2, 576, d=bf), None, None, None, 0.0, pool, 64, z(3, d=torch.int64), 1)
    with pytest.raises(ValueError):
        B.prepare_latent_gather(pool, 64, 1, z(2, 3), z(4), z(10, 576, d=bf))
    k = z(9, 4, 128, d=bf)
    with pytest.raises(ValueError):
        B.prepare_latent_prefill(z(5, 4, 192, d=bf), k, z(8, 64, d=bf), k, z(2), z(2), 0.1)
    with pytest.raises(ValueError):
        B.prepare_latent_prefill(z(5, 4, 192, d=bf), k, z(9, 64, d=bf), k, z(2), z(3), 0.1)
    # tensors of the right shape that are not on a device
    with pytest.raises(ValueError):
        B.prepare_latent_gather(pool, 64, 1, z(2, 3), z(3), z(10, 576, d=bf))


def test_workspace_size_of_nothing():
    f = B.lib().idx_latent_attention_workspace_size
    g = B.lib().idx_latent_prefill_workspace_size
    assert g(0, 999, 64) == 0 and g(4, 999, 0) == 0 and g(9, 64, 4) == 0 and g(1, 999, 1) > 0
    assert f(0, 64, 999) == 0 and f(4, 0, 999) == 0 and f(4, 64, 64) == 0 and isinstance(f(1, 1, 999), int) and ctypes.sizeof(ctypes.c_size_t) == 8
