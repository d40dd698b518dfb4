"""CPU checks of the grouped-head calls: the 64-bit statements against what they must satisfy, the
refusals of the C entry points (every call here fails its host checks, so no pointer is followed),
of the binding and of the layer."""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import kv4_ref as ref
from sparse_attention_indexer_mxfp4_gb300 import GroupedDecodeStep, GroupedLayer
from sparse_attention_indexer_mxfp4_gb300 import _binding as B

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE = 0x10000
BF, I32, I64, U8, F32 = torch.bfloat16, torch.int32, torch.int64, torch.uint8, torch.float32


def test_reference_rounds_to_the_nearest_code():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 128)) * np.exp(5 * rng.standard_normal((50, 1)))
    codes, bits = ref.quantise(x)
    back, scale = ref.values(codes, bits), np.repeat(2.0 ** (bits - 127.0), 32, -1)
    # the exponent is the least that holds the group, and steps are 1/2, 1 and 2
    amax = np.abs(x).reshape(50, 4, 32).max(-1)
    assert (amax <= 6 * 2.0 ** (bits - 127.0)).all() and (amax > 3 * 2.0 ** (bits - 127.0)).all()
    y = np.abs(x) / scale
    assert (np.abs(back - x) / scale <= np.where(y < 2, 0.25, np.where(y < 4, 0.5, 1.0))).all()


def test_reference_pages():
    """A token's parts lie in the four blocks of its page, apart from every other's."""
    seen = np.zeros(ref.page_stride(3, 2), int)
    for h in range(2):
        for o in range(3):
            for a, n in ref.spans(3, 2, h, o):
                seen[a:a + n] += 1
    assert (seen[:3 * 2 * 136] == 1).all() and (seen[3 * 2 * 136:] == 0).all()
    for page, heads in ((1, 1), (3, 2), (64, 8), (100, 5)):
        assert B.kv4_page_bytes(page, heads) == ref.page_stride(page, heads)


def _caller(name, base, places):
    fn = getattr(B.lib(), name)

    def call(**kw):
        a = list(base)
        for k, v in kw.items():
            a[places[k]] = v
        return fn(*a)
    return call


def _refused(call, status, cases):
    for kw in cases:
        assert call(**kw) == status, kw


STRIDE = 64 * 8 * 136


def test_store_refusals():
    base = [FAKE, 1024, 128, FAKE, 1024, 128, 4, 8, 128, FAKE, STRIDE, 10, 64, FAKE, None]
    p = dict(k=0, kr=1, kh=2, v=3, vr=4, vh=5, T=6, G=7, D=8, pages=9, stride=10, np=11, P=12, slots=13)
    call = _caller("idx_kv4_store", base, p)
    assert call(T=0) == 0
    _refused(call, INVALID, (dict(T=-1), dict(G=0), dict(k=None), dict(v=None), dict(slots=None), dict(kh=120), dict(vh=64),
                             dict(kr=-8), dict(pages=None), dict(stride=STRIDE - 16), dict(P=0), dict(np=-1), dict(G=9),
                             dict(G=2 ** 30, P=2 ** 30)))
    _refused(call, UNSUPPORTED, (dict(D=64), dict(k=FAKE + 2), dict(v=FAKE + 8), dict(kr=1028), dict(vh=132),
                                 dict(pages=FAKE + 8), dict(stride=STRIDE + 8), dict(np=2 ** 26)))


def test_gather_refusals():
    base = [FAKE, STRIDE, 10, 64, 8, 128, FAKE, 8, 8, FAKE, None, 2, 100, FAKE, 1024, 128, FAKE, 1024, 128, None]
    p = dict(pages=0, stride=1, np=2, P=3, G=4, D=5, bt=6, bts=7, cu=9, B=11, N=12, k=13, kr=14, kh=15, v=16, vr=17, vh=18)
    call = _caller("idx_kv4_gather", base, p)
    assert call(N=0) == 0 and call(B=0) == 0
    _refused(call, INVALID, (dict(N=-1), dict(B=-1), dict(G=0), dict(bts=7), dict(kh=120), dict(vr=-8), dict(bt=None),
                             dict(cu=None), dict(k=None), dict(v=None), dict(stride=100), dict(pages=None)))
    _refused(call, UNSUPPORTED, (dict(D=256, kh=256, vh=256), dict(k=FAKE + 8), dict(vr=1020), dict(pages=FAKE + 4)))


def test_attention_refusals():
    base = [FAKE, 8192, 128, FAKE, STRIDE, 10, 64, FAKE, FAKE, 90000, 4, 64, 8, 128, 0.1, FAKE, 8192, 128, FAKE, 64, FAKE,
            1 << 40, None]
    p = dict(q=0, qr=1, qh=2, pages=3, stride=4, np=5, P=6, slots=7, indptr=8, ns=9, R=10, H=11, G=12, D=13, scale=14, out=15,
             outr=16, oh=17, ldl=19, ws=20, wsb=21)
    call = _caller("idx_kv4_attention", base, p)
    assert call(R=0) == 0
    _refused(call, INVALID, (dict(R=-1), dict(H=0), dict(G=0), dict(q=None), dict(out=None), dict(indptr=None),
                             dict(slots=None), dict(ns=-1), dict(scale=0.0), dict(scale=float("nan")),
                             dict(scale=float("inf")), dict(qh=120), dict(oh=64), dict(ldl=63), dict(stride=STRIDE - 16),
                             dict(qr=-8), dict(pages=None)))
    _refused(call, UNSUPPORTED, (dict(H=63), dict(D=64), dict(q=FAKE + 2), dict(qr=8196), dict(out=FAKE + 8), dict(outr=4),
                                 dict(pages=FAKE + 8), dict(ns=2 ** 31), dict(R=2 ** 30)))
    _refused(call, WORKSPACE, (dict(ws=None), dict(wsb=0), dict(ws=FAKE + 8)))


def test_paged_refusals():
    base = [FAKE, 8192, 128, FAKE, STRIDE, 10, 64, FAKE, 1600, FAKE, 0, 2, 2, 100000, 64, 8, 128, 0.1, FAKE, 8192, 128, None,
            0, FAKE, 1 << 40, None]
    p = dict(q=0, bt=7, bts=8, ctx=9, B=11, n=12, mml=13, H=14, G=15, out=18, ws=23, wsb=24)
    call = _caller("idx_paged_kv4_attention", base, p)
    assert call(B=0) == 0
    _refused(call, INVALID, (dict(B=-1), dict(n=0), dict(mml=-1), dict(bts=1562), dict(bt=None), dict(ctx=None), dict(q=None)))
    _refused(call, UNSUPPORTED, (dict(B=2 ** 30, n=4), dict(H=20), dict(out=FAKE + 2)))
    assert call(wsb=0) == WORKSPACE


def test_weights_refusals():
    base = [FAKE, 8192, 128, FAKE, STRIDE, 10, 64, FAKE, 16, FAKE, 0, 2, 2, 1000, 64, 8, 128, 0.1, FAKE, 64, 1, FAKE, 9000,
            1000, 1000, FAKE + 64, 9000, 1000, None]
    p = dict(q=0, bts=8, ctx=9, B=11, n=12, mml=13, H=14, lse=18, ldl=19, ldlh=20, mass=21, lb=22, lh=23, width=24, out=25,
             ob=26, oh=27)
    call = _caller("idx_paged_kv4_weights", base, p)
    assert call(B=0) == 0
    _refused(call, INVALID, (dict(B=-1), dict(n=0), dict(width=999), dict(bts=15), dict(lse=None), dict(ldl=-1),
                             dict(ldlh=-1), dict(out=None), dict(lb=-1), dict(oh=-1), dict(mass=FAKE + 64, lb=9001)))
    _refused(call, UNSUPPORTED, (dict(H=20), dict(q=FAKE + 4), dict(B=2 ** 30, n=4)))


def test_evict_refusals():
    base = [FAKE, 9000, 1000, 1000, FAKE, 2, 8, 128, 100, 10, 0, FAKE, STRIDE, 10, 64, FAKE, 16, 16, FAKE, 2, 2, FAKE, FAKE,
            FAKE, FAKE, 1 << 30, None]
    p = dict(mass=0, lb=1, lh=2, ld=3, ctx=4, B=5, G=6, D=7, budget=8, recent=9, whole=10, pages=11, stride=12, P=14, bt=15,
             bts=16, mb=17, nt=18, nts=19, nb=20, keep=21, lens=22, nm=23, ws=24, wsb=25)
    call = _caller("idx_kv4_evict", base, p)
    assert call(B=0) == 0
    _refused(call, INVALID, (dict(B=-1), dict(G=0), dict(ld=-1), dict(budget=-1), dict(recent=-1), dict(recent=101),
                             dict(mass=None), dict(ctx=None), dict(bts=15), dict(nts=1), dict(nb=1), dict(bt=None),
                             dict(nt=None), dict(keep=None), dict(lens=None), dict(nm=None), dict(pages=None),
                             dict(stride=100), dict(lh=-1)))
    _refused(call, UNSUPPORTED, (dict(D=64), dict(B=60000), dict(pages=FAKE + 8)))
    _refused(call, WORKSPACE, (dict(ld=300000, ws=None), dict(ld=300000, wsb=8), dict(ld=300000, ws=FAKE + 8)))


def test_grouped_prefill_refusals():
    base = [FAKE, 8192, 128, FAKE, 1024, 128, FAKE, 1024, 128, FAKE, FAKE, 2, 100, 1000, 64, 8, 128, 0.1, 1, FAKE, 8192, 128,
            FAKE, 64, FAKE, 1 << 30, None]
    p = dict(q=0, qr=1, qh=2, k=3, kr=4, kh=5, v=6, vr=7, vh=8, cq=9, ck=10, B=11, Tq=12, Tk=13, H=14, G=15, D=16, scale=17,
             out=19, outr=20, oh=21, ldl=23, ws=24, wsb=25)
    call = _caller("idx_grouped_prefill", base, p)
    assert call(B=0) == 0 and call(Tq=0) == 0
    _refused(call, INVALID, (dict(B=-1), dict(Tq=-1), dict(Tk=-1), dict(H=0), dict(G=0), dict(q=None), dict(k=None),
                             dict(v=None), dict(cq=None), dict(ck=None), dict(out=None), dict(scale=-1.0), dict(qh=64),
                             dict(kh=64), dict(vh=64), dict(oh=64), dict(ldl=63), dict(qr=-8)))
    _refused(call, UNSUPPORTED, (dict(D=64), dict(G=7), dict(q=FAKE + 2), dict(kr=1028), dict(v=FAKE + 8),
                                 dict(H=65544, ldl=65544)))
    _refused(call, WORKSPACE, (dict(ws=None), dict(wsb=0), dict(ws=FAKE + 8)))


def test_scratch_of_nothing():
    L = B.lib()
    f, g, e = L.idx_kv4_attention_workspace_size, L.idx_grouped_prefill_workspace_size, L.idx_kv4_evict_workspace_size
    assert f(0, 1, 64, 8, 9999) == 0 and f(400, 1, 64, 8, 512) == 0 and f(400, 1, 64, 8, 513) > 0
    assert f(400, 4, 64, 8, 513) > f(400, 1, 64, 8, 513)  # wider blocks of columns
    assert g(0, 999, 64) == 0 and g(4, 512, 64) == 0 and g(4, 513, 64) > 0
    # what a cluster holds needs none
    n = 1 << 19
    assert e(0, 8, n, 9, 1, 0) == 0 and e(2, 8, n, n, 1, 0) == 0 and e(2, 8, n, 9, 9, 0) == 0
    assert e(2, 8, 262144, 9, 1, 0) == 0 and e(2, 8, n, 9, 1, 0) > e(2, 8, n, 9, 1, 1) > 0


# ------------------------------------------------------------------- the binding


def _z(*shape, d=I32):
    return torch.zeros(*shape, dtype=d)


def _pool():
    return _z(4, B.kv4_page_bytes(64, 2), d=U8)


CALLS = {
    "prefill": (B.idx_grouped_prefill, B.prepare_grouped_prefill,
                lambda: [_z(5, 4, 128, d=BF), _z(8, 2, 128, d=BF), _z(8, 2, 128, d=BF), _z(2), _z(2), 0.1]),
    "store": (B.idx_kv4_store, B.prepare_kv4_store,
              lambda: [_z(3, 2, 128, d=BF), _z(3, 2, 128, d=BF), _pool(), 64, _z(3, d=I64)]),
    "gather": (B.idx_kv4_gather, B.prepare_kv4_gather,
               lambda: [_pool(), 64, _z(2, 3), _z(3), _z(9, 2, 128, d=BF), _z(9, 2, 128, d=BF), _z(2)]),
    "attention": (B.idx_kv4_attention, B.prepare_kv4_attention,
                  lambda: [_z(3, 4, 128, d=BF), _pool(), 64, 2, _z(5), _z(4), 0.1]),
    "paged": (B.idx_paged_kv4_attention, B.prepare_paged_kv4_attention,
              lambda: [_z(4, 4, 128, d=BF), _pool(), 64, 2, _z(2, 3), _z(2), 2, 0.1, 192]),
    "weights": (B.idx_paged_kv4_weights, B.prepare_paged_kv4_weights,
                lambda: [_z(4, 4, 128, d=BF), _pool(), 64, 2, _z(2, 3), _z(2), 2, 0.1, 192, _z(4, 4, d=F32),
                         _z(2, 2, 192, d=F32)]),
    "evict": (B.idx_kv4_evict, B.prepare_kv4_evict,
              lambda: [_z(2, 2, 192, d=F32), _z(2), 64, 8, _pool(), 64, _z(2, 3), _z(2, 1)]),
}
# (call, argument, what is put in its place)
WRONG = [
    ("prefill", 0, _z(5, 3, 128, d=BF)), ("prefill", 1, _z(7, 2, 128, d=BF)), ("prefill", 1, _z(8, 2, 128, d=F32)),
    ("prefill", 2, _z(8, 1, 128, d=BF)), ("prefill", 3, _z(3)), ("prefill", 4, _z(2, d=I64)), ("prefill", 0, None),
    ("store", 0, _z(3, 2, 64, d=BF)), ("store", 1, _z(3, 1, 128, d=BF)), ("store", 2, _z(4, 64)), ("store", 4, _z(3)),
    ("store", 4, _z(4, d=I64)), ("store", 3, 1 << 40),
    ("gather", 0, None), ("gather", 2, _z(1, 3)), ("gather", 3, _z(0)), ("gather", 3, _z(3, d=I64)),
    ("gather", 4, _z(9, 2, 128, d=F32)), ("gather", 5, _z(8, 2, 128, d=BF)), ("gather", 6, _z(3)),
    ("attention", 0, _z(3, 128, d=BF)), ("attention", 3, 3), ("attention", 3, 0), ("attention", 4, _z(5, d=I64)),
    ("attention", 4, _z(10)[::2]), ("attention", 5, _z(5)),
    ("paged", 4, _z(6)), ("paged", 4, _z(1, 3)), ("paged", 5, _z(4)), ("paged", 6, 3), ("paged", 6, 0), ("paged", 3, -1),
    ("weights", 9, _z(4, 3, d=F32)), ("weights", 9, _z(4, 4, d=BF)), ("weights", 10, _z(2, 2, 191, d=F32)),
    ("weights", 10, _z(2, 1, 192, d=F32)), ("weights", 10, _z(2, 192, d=F32)),
    ("evict", 0, _z(2, 192, d=F32)), ("evict", 0, _z(2, 2, 192, d=BF)), ("evict", 1, _z(3)), ("evict", 2, 7),
    ("evict", 3, -1), ("evict", 3, 65), ("evict", 6, _z(1, 3)), ("evict", 7, _z(2, 0)), ("evict", 7, _z(1, 1)),
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


@pytest.mark.parametrize("name,given", [
    ("attention", dict(out=_z(3, 4, 120, d=BF))), ("attention", dict(lse=_z(3, 4))), ("paged", dict(out=_z(3, 4, 128, d=BF))),
    ("prefill", dict(lse=_z(2, 4, d=F32))), ("paged", dict(workspace=_z(64, d=U8)[::2])),
    ("weights", dict(out=_z(2, 2, 193, d=F32))), ("evict", dict(keep=_z(2, 2, 63))), ("evict", dict(new_lens=_z(2, d=I64))),
    ("evict", dict(new_mass=_z(2, 64, 2, d=F32))), ("evict", dict(whole_tokens=True, keep=_z(2, 2, 64))),
    ("evict", dict(workspace=_z(64, d=U8)[::2]))])
def test_wrong_outputs(name, given):
    call, prepare, good = CALLS[name]
    for f in (call, prepare):
        with pytest.raises(ValueError):
            f(*good(), **given)


# --------------------------------------------------------------------- the layer


def test_layer_refusals():
    for heads, kv in ((4, 3), (4, 0), (0, 1)):
        with pytest.raises(ValueError, match="kv_heads"):
            GroupedLayer(heads, kv, 4, 64, device="cpu")
    layer = GroupedLayer(4, 2, 4, 64, device="cpu")
    with pytest.raises(ValueError, match="rows, 4"):
        layer.decode_slots(_z(3, 8, 128, d=BF), _z(5), _z(4))
    with pytest.raises(ValueError, match="tokens, 2"):
        layer.store(_z(3, 4, 128, d=BF), _z(3, 4, 128, d=BF), _z(3, d=I64))
    with pytest.raises(ValueError, match="mass"):
        layer.evict(_z(2, 1, 99, d=F32), _z(2), 10, 1, _z(2, 3), _z(2, 1))
    for page_size, pages in ((16, 4), (64, 5)):
        with pytest.raises(ValueError, match="pages"):
            GroupedDecodeStep(SimpleNamespace(page_size=page_size, num_pages=pages), layer, _z(2, 4, 128, d=BF), device="cpu")
