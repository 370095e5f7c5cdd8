"""The steps of a verification round in 64 bits, written from their
definitions in include/svw.h, with the error bounds that the tests use."""
import numpy as np

F32 = 2.0 ** -24   # half an ulp of fp32, relative
BF16 = 2.0 ** -8   # half an ulp of bf16, relative


def adjust(x, cu, tokens, history, cu_h, prompt, rep, freq, pres, biases, mask, mask_row, bonus):
    """x: float64 [rows, V]; biases: per request a list of (token, value) in
    order; mask: bool [mask rows, V] or None.  Returns (y, size): size bounds
    the intermediate values of each entry."""
    y, size = x.copy(), np.abs(x)
    N = len(cu) - 1
    for i in range(N):
        hist = history[cu_h[i]:cu_h[i + 1]]
        p = prompt[i]
        for j in range(cu[i + 1] - cu[i] + (1 if bonus else 0)):
            r = cu[i] + j + (i if bonus else 0)
            said = list(hist[p:]) + list(tokens[cu[i]:cu[i] + j])
            n = np.bincount(said, minlength=x.shape[1]) if said else np.zeros(x.shape[1], np.int64)
            seen = n > 0
            seen[hist[:p]] = True
            row = x[r].copy()
            with np.errstate(invalid="ignore"):
                row[seen] = np.where(row[seen] > 0, row[seen] / rep[i], row[seen] * rep[i])
            s = np.maximum(np.abs(x[r]), np.abs(row))
            row = np.where(n > 0, row - freq[i] * n - pres[i], row)
            s += abs(freq[i]) * n + abs(pres[i]) * (n > 0)
            for v, b in dict(biases[i]).items():  # the last one listed
                row[v] += b
                s[v] += abs(b) if np.isfinite(b) else 0
            if mask is not None and mask_row[r] >= 0:
                row[~mask[mask_row[r]]] = -np.inf
            y[r], size[r] = row, s
    return y, size


def adjust_bound(y, size, bf16):
    """At most four fp32 roundings of values bounded by size, then one to bf16."""
    y = np.where(np.isfinite(y), np.abs(y), 0)
    size = np.where(np.isfinite(size), size, 0)
    return 4.01 * F32 * size + (1.01 * BF16 * (y + 4.01 * F32 * size) if bf16 else 0)


def rotate(x, cs, rot, interleaved):
    """x: float64 [tokens, heads, dim], cs: float64 [tokens, rot].  Returns (y, size)."""
    y, size = x.copy(), np.zeros_like(x)
    h = rot // 2
    u = np.arange(h)
    a, b = (2 * u, 2 * u + 1) if interleaved else (u, u + h)
    c, s = cs[:, None, :h], cs[:, None, h:]
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
    size[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, size


def rotate_bound(y, size, bf16):
    """Two rounded products and a rounded sum, then one rounding to bf16."""
    return 2.01 * F32 * size + (1.01 * BF16 * (np.abs(y) + 2.01 * F32 * size) if bf16 else 0)


def attend(q, k, v, scale, causal, window):
    """One request and one query head: q [n, D], k, v [kv, D] float64.  Returns
    (out, lse, out_bound, lse_bound)."""
    n, kv = q.shape[0], k.shape[0]
    at = kv - n + np.arange(n)[:, None]
    j = np.arange(kv)[None]
    ok = np.ones((n, kv), bool)
    if causal:
        ok = j <= at
        if window:
            ok &= j > at - window
    x = scale * (q @ k.T)
    x = np.where(ok, x, -np.inf)
    some = ok.any(1)
    m = np.where(some, x.max(1, initial=-np.inf), 0.0)
    e = np.exp(x - m[:, None])
    total = e.sum(1)
    w = e / np.where(some, total, 1.0)[:, None]
    out = w @ v
    with np.errstate(divide="ignore"):
        lse = m + np.log(total)
    # a score: exact products, D of them summed in fp32 (each step may also be
    # cut instead of rounded: one ulp), scaled by a rounded factor, the maximum
    # subtracted; its exponential within 2^-22
    D = q.shape[1]
    eps = ((D + 8) * 2 * F32 * scale * (np.abs(q) @ np.abs(k).T) * ok).max(1, initial=0.0) + 2.0 ** -21
    eps_sum = (kv / 16 + 64) * F32  # partial sums of a row
    mass = w @ np.abs(v)
    acc = (kv / 8 + 64) * 2 * F32  # the second product, summed in fp32
    out_bound = (1.01 * BF16 + 2 * eps + eps_sum + acc)[:, None] * mass + 1.01 * BF16 * np.abs(out) + 1e-30
    lse_bound = 2 * eps + eps_sum + 4 * F32 * np.abs(np.where(some, lse, 0))
    return out, lse, out_bound, lse_bound
