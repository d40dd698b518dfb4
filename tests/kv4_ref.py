"""Plain 64-bit statements of the 4-bit cache and of what the calls over it compute."""
import numpy as np

from latent_ref import HALF_BF16, attend  # noqa: F401

D, GROUP = 128, 32
VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
HALF_F16 = 2.0 ** -11


def page_stride(page, heads, extra=0):
    return -(-page * heads * 136 // 16) * 16 + extra


def spans(page, heads, head, off):
    """(first byte, bytes) of a head's token in its page: codes of K and V, scales of K and V."""
    n = page * heads
    at = head * page + off
    return [(at * 64, 64), (n * 64 + at * 64, 64), (n * 128 + at * 4, 4), (n * 132 + at * 4, 4)]


def quantise(x):
    """(codes [..., 128], scale bytes [..., 4]) of finite x, by the store's definition."""
    y = np.asarray(x, np.float64).reshape(*x.shape[:-1], 4, GROUP)
    amax = np.maximum(np.abs(y).max(-1, keepdims=True), 2.0 ** -126)
    m, e = np.frexp(amax / 6)  # in [1/2, 1): the power above it, or itself where it is one
    bits = np.clip(np.where(m == 0.5, e - 1, e) + 127, 0, 254)
    z = np.abs(y) * 2.0 ** (127.0 - bits)
    gap = np.abs(z[..., None] - VALUES)
    best = gap.min(-1, keepdims=True)
    tie = gap == best
    even = tie & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), tie.argmax(-1))
    code = code | (np.signbit(y).astype(int) << 3)
    return code.reshape(x.shape).astype(np.uint8), bits[..., 0].astype(np.uint8)


def values(codes, bits):
    v = VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(bits == 255, np.nan, 2.0 ** (bits.astype(float) - 127))
    return v * np.repeat(s, GROUP, -1)


def write(pool, page, heads, slot, head, side, codes, bits):
    line, s = pool[slot // page], spans(page, heads, head, slot % page)
    (a, n), (b, k) = s[side], s[2 + side]
    line[a:a + n] = codes[::2] | codes[1::2] << 4
    line[b:b + k] = bits


def read(pool, page, heads, slots, head):
    """K and V [n, 128] of a head's tokens."""
    out = np.zeros((2, len(slots), D))
    for i, slot in enumerate(slots):
        line, s = pool[slot // page], spans(page, heads, head, slot % page)
        for side in range(2):
            (a, n), (b, k) = s[side], s[2 + side]
            byte = line[a:a + n]
            codes = np.stack([byte & 15, byte >> 4], -1).reshape(-1)
            out[side, i] = values(codes, line[b:b + k])
    return out


def make_pool(rng, pages, page, heads, extra=0, spread=1.0):
    """Random codes; scales around 1/4, over `spread` powers of two either way."""
    pool = rng.integers(0, 256, (pages, page_stride(page, heads, extra)), dtype=np.uint8)
    n = page * heads
    e = rng.integers(-int(spread), int(spread) + 1, (pages, n * 8)) + 125
    pool[:, n * 128:n * 136] = e.astype(np.uint8)
    return pool


def poison(pool, page, heads, used):
    """Tokens outside the used slots become NaN (their scales)."""
    keep = np.zeros(pool.shape[0] * page, bool)
    keep[np.asarray(used, np.int64)] = True
    for s in np.flatnonzero(~keep):
        for h in range(heads):
            for a, n in spans(page, heads, h, s % page)[2:]:
                pool[s // page, a:a + n] = 255


def check(out, lse, ref, keys, weight=HALF_F16, vmax=0.0):
    """A weight is off by its rounding (half a step of f16, or of bf16) and by the error of its
    score, the result by its own rounding to bf16.  A score is a sum of 128 exact products in 32
    bits and a scaling: off by at most 136 * 2^-23 of the sum of their magnitudes; the
    exponential adds a few units of 2^-22.  f16 weights are held from 2^-24 on, 2^6 times
    larger and under a maximum that may be 2^4 too low: 2^-26 of the largest value each."""
    o, l, pv, mag = ref
    ds = 136 * 2.0 ** -23 * mag + 2.0 ** -20
    tol = HALF_BF16 * np.abs(o) + (weight * 1.01 + 2 * ds[:, None]) * pv * (1 + HALF_BF16) + keys * 2.0 ** -26 * vmax + 1e-30
    assert np.isfinite(out).all()
    bad = np.abs(out - o) - tol
    assert (bad <= 0).all(), f"out is off by {np.abs(out - o).max()}, {bad.max()} over its bound"
    if lse is not None:
        fin = np.isfinite(l)
        assert np.array_equal(fin, np.isfinite(lse)) and (lse[~fin] == -np.inf).all()
        err = np.abs(lse[fin] - l[fin])
        assert (err <= 2 * ds[fin] + 2.0 ** -22 * np.abs(l[fin])).all(), err.max()
