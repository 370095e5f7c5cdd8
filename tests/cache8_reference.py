"""The calls of an 8-bit cache in 64 bits, written from their definitions in
include/svw.h, with the error bounds that the tests use."""
import numpy as np

import round_reference as ref
from round_reference import BF16, F32


def nearest(x):
    """The nearest of e4m3's values, the even one of two: steps of 2^-3 of the
    power of two below, 2^-9 at least; +-448 beyond them."""
    x = np.asarray(x, np.float64)
    ok = np.where(np.isfinite(x), x, 0.0)
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(ok), 2.0 ** -60))), -6)
    step = 2.0 ** (e - 3)
    y = np.clip(np.round(ok / step) * step, -448, 448)  # a value that rounds up to a power of two is its multiple too
    return np.where(np.isnan(x), np.nan, np.where(np.isinf(x), np.sign(x) * 448, y))


def norm(x, weight, eps):
    """x: float64 [..., dim].  Returns (y, bound): r's sum of dim squares and its
    root, then two products, in fp32."""
    if weight is None:
        return x, np.zeros_like(x)
    d = x.shape[-1]
    y = x * weight / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y, np.abs(y) * (d / 2 + 12) * F32


def rotate(y, err, cs, rot, interleaved):
    """The rotation of values known to within err: (z, bound)."""
    z, size = ref.rotate(y, cs, rot, interleaved)
    h = rot // 2
    u = np.arange(h)
    a, b = (2 * u, 2 * u + 1) if interleaved else (u, u + h)
    c, s = np.abs(cs[:, None, :h]), np.abs(cs[:, None, h:])
    carried = err.copy()
    carried[..., a] = err[..., a] * c + err[..., b] * s
    carried[..., b] = err[..., b] * c + err[..., a] * s
    return z, carried + 2.01 * F32 * size


def code_range(z, err, scale):
    """The least and the greatest code that z / scale, z within err, may have: a
    rounded reciprocal and product, then the nearest code."""
    x, e = z / scale, err / scale
    e = e + 3.01 * F32 * (np.abs(x) + e)
    return nearest(x - e), nearest(x + e)


def attend(q, k, v, scale, causal, window):
    """round_reference's attend, its bounds widened by the roundings of queries and
    weights to two codes."""
    out, lse, ob, lb = ref.attend(q, k, v, scale, causal, window)
    n, kv = q.shape[0], k.shape[0]
    most = np.abs(q).max(1, keepdims=True)
    # a query's elements below 2^-10 of its largest: within 2^-17 of that one
    q_err = np.where(np.abs(q) < 2.0 ** -10 * most, 2.0 ** -17 * most, 0.0)
    at = kv - n + np.arange(n)[:, None]
    j = np.arange(kv)[None]
    ok = np.ones((n, kv), bool)
    if causal:
        ok = j <= at
        if window:
            ok &= j > at - window
    eps = (scale * (q_err @ np.abs(k).T) * ok).max(1, initial=0.0)
    x = np.where(ok, scale * (q @ k.T), -np.inf)
    with np.errstate(invalid="ignore"):
        w = np.where(ok, np.exp(x - np.where(np.isfinite(lse), lse, 0)[:, None]), 0.0)
    # a weight: fp16's 2^-11, then the nearest code (2^-4) and the nearest one of the rest (2^-4 of it): 2^-8, as
    # bf16; within 2^-15 of the largest at least
    more = 2.0 ** -11 * 1.01 * (w @ np.abs(v)) + 2.0 ** -15 * w.max(1, initial=0.0)[:, None] * (ok @ np.abs(v))
    return out, lse, ob + 2 * eps[:, None] * (w @ np.abs(v)) + 1.01 * more, lb + 2 * eps
