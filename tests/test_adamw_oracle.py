"""Pins of the oracle of the AdamW step: closed forms, the grids of 8-bit floats
as torch's own casts have them, and unbiased rounding."""

import numpy as np
import pytest
import torch

from oracle import train_ops as T


def test_first_step_is_the_sign_of_the_gradient():
    g = np.array([3.0, -0.5, 1e-3])
    m, v = T.adamw_moments(np.zeros(3), np.zeros(3), g, 0.9, 0.999)
    w = T.adamw_weights(np.ones(3), m.astype(float), v.astype(float), 1, 0.1, 0.9, 0.999, 1e-12, 0.0)
    assert np.allclose(w, 1 - 0.1 * np.sign(g), atol=1e-6)
    w = T.adamw_weights(np.ones(3), m * 0.0, v.astype(float), 1, 0.1, 0.9, 0.999, 1e-12, 0.5)
    assert np.allclose(w, 1 - 0.1 * 0.5)


def test_matches_torchs_optimizer_over_steps():
    r = np.random.default_rng(0)
    w0, grads = r.standard_normal(50), r.standard_normal((7, 50))
    p = torch.nn.Parameter(torch.from_numpy(w0.copy()))
    opt = torch.optim.AdamW([p], lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    w, m, v = w0.copy(), np.zeros(50), np.zeros(50)
    for t, g in enumerate(grads, 1):
        p.grad = torch.from_numpy(g.copy())
        opt.step()
        m, v = 0.8 * m + 0.2 * g, 0.95 * v + 0.05 * g * g
        w = T.adamw_weights(w, m, v, t, 0.01, 0.8, 0.95, 1e-6, 0.1)
    assert np.allclose(w, p.detach().numpy(), rtol=1e-9)


@pytest.mark.parametrize("digits,bias,top,kind", [(3, 7, 7, torch.float8_e4m3fn), (2, 15, 14, torch.float8_e5m2)])
def test_codes_are_those_of_the_type(digits, bias, top, kind):
    """Every finite value of the type below 2^(top + 1) is kept whatever the random bits; between two, r decides."""
    grid = torch.arange(128, dtype=torch.uint8).view(kind).double().numpy()
    grid = grid[np.isfinite(grid) & (grid < 2.0 ** (top + 1))]
    assert grid[-1] >= 2.0 ** top
    x = np.concatenate([grid, -grid]).astype(np.float32)[None]
    x = np.pad(x, ((0, 0), (0, 256 - x.size)))[0]
    for r in (0, 65535):
        q, s = T.encode8(x, np.full(256, r), digits, bias, top)
        assert s[0] == 1.0 and np.array_equal(q, x)
    for a, b in ((5, 6), (40, 41), (1, 2), (0, 1)):
        lo, hi = grid[a], grid[b]
        x = np.zeros(256, dtype=np.float32)
        x[0], x[1] = grid[-1], lo + 0.25 * (hi - lo)
        r = np.zeros(256, dtype=np.int64)
        for bits, want in ((0, lo), (49151, lo), (49152, hi), (65535, hi)):
            r[1] = bits
            assert T.encode8(x, r, digits, bias, top)[0][1] == want


def test_rounding_is_unbiased():
    x = np.random.default_rng(1).standard_normal(256).astype(np.float32) * 1e-3
    total = np.zeros(256)
    for n in range(64):   # a grid of 64 equally spread random numbers: the mean is off by 1 / 64 of a step at most
        total += T.encode8(x, np.full(256, n * 1024 + 512), 3, 7, 7)[0]
    step = np.maximum(np.abs(x), 2.0 ** -6 * 2.0 ** -17) / 8
    assert (np.abs(total / 64 - x) <= step / 64).all()


def test_values_that_are_not_finite():
    x = np.array([np.nan, np.inf, -np.inf, 1.0] + [0.0] * 252, dtype=np.float32)
    q, s = T.encode8(x, np.zeros(256, dtype=np.int64), 3, 7, 7)
    assert np.isnan(q[:3]).all() and q[3] == 1.0 and s[0] == 2.0 ** -7
    q, s = T.encode8(np.zeros(300, dtype=np.float32), np.full(300, 65535), 2, 15, 14)
    assert not q.any() and (s == 2.0 ** -120).all()


def test_random_bits_repeat_by_counter():
    a = T.random16(100, 3, 1 << 40, 7)
    assert np.array_equal(a[:37], T.random16(37, 3, 1 << 40, 7))
    assert not np.array_equal(a, T.random16(100, 4, 1 << 40, 7))
    assert a.min() >= 0 and a.max() < 65536
