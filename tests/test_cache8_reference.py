"""The 64-bit reference of an 8-bit cache against torch's own conversions."""
import numpy as np
import torch

import cache8_reference as c8


def test_nearest_is_the_nearest_code():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    finite = np.sort(codes[np.isfinite(codes)])
    assert np.array_equal(c8.nearest(finite), finite)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=4000) * 10.0 ** rng.uniform(-4, 2.5, 4000), (finite[1:] + finite[:-1]) / 2])
    far = np.abs(x[:, None] - finite[None])
    assert np.array_equal(np.abs(x - c8.nearest(x)), far.min(1))
    inside = x[np.abs(x) <= 448].astype(np.float32)
    want = torch.from_numpy(inside).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(c8.nearest(inside.astype(np.float64)), want)
    assert np.array_equal(c8.nearest([1e9, -1e9, np.inf, -np.inf]), [448, -448, 448, -448])
    assert np.isnan(c8.nearest([np.nan])).all()


def test_norm_and_rotation():
    rng = np.random.default_rng(1)
    x, w = rng.normal(size=(3, 2, 8)), rng.normal(size=8)
    y, _ = c8.norm(x, w, 1e-5)
    assert np.allclose(y, x / np.sqrt((x ** 2).sum(-1, keepdims=True) / 8 + 1e-5) * w)
    a = rng.uniform(0, 6, size=(3, 3))
    cs = np.concatenate([np.cos(a), np.sin(a)], 1)
    z, bound = c8.rotate(y, np.abs(y) * 1e-3, cs, 6, True)
    assert np.allclose((z[..., :6] ** 2).sum(-1), (y[..., :6] ** 2).sum(-1)) and np.array_equal(z[..., 6:], y[..., 6:])
    near, _ = c8.rotate(y * (1 + 1e-3 * rng.uniform(-1, 1, y.shape)), np.zeros_like(y), cs, 6, True)
    assert np.all(np.abs(near - z) <= bound)
