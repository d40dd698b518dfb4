"""Plain 64-bit statements of the latent cache and its attention (numpy, no
library code), and the tolerances that follow from the kernels' roundings."""
import numpy as np
import torch

L, ROPE, GROUP, TOK = 512, 64, 64, 576
BF16, FP8 = 0, 1
HALF_BF16 = 2.0 ** -8  # torch.finfo(torch.bfloat16).eps / 2


def token_bytes(fmt):
    return 2 * TOK if fmt == BF16 else L + 2 * ROPE + L // GROUP


def page_stride(fmt, page, extra=0):
    return -(-page * token_bytes(fmt) // 16) * 16 + extra


def bf16_float(raw):
    """uint8 [..., 2 n] -> float64 [..., n], little-endian bf16."""
    u = np.ascontiguousarray(raw).view(np.uint16).astype(np.uint32) << 16
    return u.view(np.float32).astype(np.float64)


def e4m3_float(raw):
    b = raw.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(b >> 7, -v, v)


def read_tokens(pool, fmt, page, slots):
    """float64 [n, 576] of the tokens in these slots (all inside the pool)."""
    out = np.empty((len(slots), TOK))
    for i, s in enumerate(np.asarray(slots, np.int64)):
        line, o = pool[s // page], s % page
        if fmt == BF16:
            out[i] = bf16_float(line[o * 1152:(o + 1) * 1152])
            continue
        code = e4m3_float(line[o * L:(o + 1) * L]).reshape(L // GROUP, GROUP)
        r0, s0 = page * L, page * (L + 2 * ROPE)
        bits = line[s0 + o * 8:s0 + o * 8 + 8].astype(np.float64)
        scale = np.where(bits == 255, np.nan, 2.0 ** (bits - 127))
        out[i, :L] = (code * scale[:, None]).reshape(-1)
        out[i, L:] = bf16_float(line[r0 + o * 128:r0 + (o + 1) * 128])
    return out


def make_pool(rng, fmt, pages, page, extra=0, spread=1.0):
    """A pool of plausible tokens, as bytes (uint8 [pages, stride])."""
    stride = page_stride(fmt, page, extra)
    pool = rng.integers(0, 256, (pages, stride), dtype=np.uint8)
    x = rng.standard_normal((pages, page, TOK)) * np.exp(spread * rng.standard_normal((pages, page, 1)))
    bf = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint8)
    if fmt == BF16:
        pool[:, :page * 1152] = bf.reshape(pages, -1)
        return pool
    y = x[..., :L].reshape(pages, page, L // GROUP, GROUP)
    bits = np.ceil(np.log2(np.abs(y).max(-1, keepdims=True) / 448.0)) + 127
    code = torch.from_numpy((y * 2.0 ** (127 - bits)).astype(np.float32)).to(torch.float8_e4m3fn)
    pool[:, :page * L] = code.view(torch.uint8).numpy().reshape(pages, -1)
    pool[:, page * L:page * 640] = bf.reshape(pages, page, 1152)[..., 1024:].reshape(pages, -1)
    pool[:, page * 640:page * 648] = bits.astype(np.uint8).reshape(pages, -1)
    return pool


def poison(pool, fmt, page, used):
    """Everything outside the used slots becomes NaN (codes, scales and bf16)."""
    keep = np.zeros(pool.shape[0] * page, bool)
    keep[np.asarray(used, np.int64)] = True
    for s in np.flatnonzero(~keep):
        line, o = pool[s // page], s % page
        if fmt == BF16:
            line[o * 1152:(o + 1) * 1152] = 0xff
        else:
            line[o * L:(o + 1) * L] = 0x7f
            line[page * L + o * 128:page * L + (o + 1) * 128] = 0xff
            line[page * 640 + o * 8:page * 640 + (o + 1) * 8] = 0xff


def attend(q, k, v, scale, seen=None):
    """q [n, d], k [m, d], v [m, e]: out [n, e], lse [n], and the sums of p |v|
    and the largest sum of |q k| that the tolerances need."""
    s = q @ k.T * scale
    if seen is not None:
        s = np.where(seen, s, -np.inf)
    if s.shape[1] == 0:
        z = np.zeros((q.shape[0], v.shape[1]))
        return z, np.full(q.shape[0], -np.inf), z, np.zeros(q.shape[0])
    top = s.max(1, keepdims=True)
    p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    tot = p.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (np.log(tot) + np.where(np.isfinite(top), top, 0.0))[:, 0]
    p = p / np.where(tot == 0, 1.0, tot)
    return p @ v, lse, p @ np.abs(v), (np.abs(q) @ np.abs(k).T).max(1) * scale


def check(out, lse, ref):
    """A weight is off by its rounding to bf16 (half a step) and by the error of
    its score, the result by its own rounding.  A score is a sum of at most 576
    exact products in 32 bits: off by at most 576 * 2^-23 of the sum of their
    magnitudes, and the exponential adds a few units of 2^-22."""
    o, l, pv, mag = ref
    ds = 576 * 2.0 ** -23 * mag + 2.0 ** -20
    tol = HALF_BF16 * np.abs(o) + (HALF_BF16 * 1.01 + 2 * ds[:, None]) * pv + 1e-30
    assert np.isfinite(out).all()
    bad = np.abs(out - o) - tol
    assert (bad <= 0).all(), f"out is off by {np.abs(out - o).max()}, {bad.max()} over its bound"
    if lse is not None:
        fin = np.isfinite(l)
        assert np.array_equal(fin, np.isfinite(lse)) and (lse[~fin] == -np.inf).all()
        err = np.abs(lse[fin] - l[fin])
        assert (err <= 2 * ds[fin] + 2.0 ** -22 * np.abs(l[fin])).all(), err.max()
