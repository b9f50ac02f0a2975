"""8-bit moments of gradients that differ widely within a block: the oracle's many steps (no GPU).

Exact moments cannot make a step longer than
  (1 - b1) / (1 - b1^t) sqrt((1 - b2^t) / (1 - b2)) sqrt(sum_{k < t} (b1^2 / b2)^k) lr
whatever the gradients (Cauchy and Schwarz, m as a sum of g_i sqrt(b2)^(t - i) times the rest). A code is off by at
most a step of its type, 1 / 8 of m up and 1 / 4 of v down, which leaves 1.125 / sqrt(3 / 4) < 1.3 times that."""

import numpy as np
import pytest

from oracle import train_ops as T

SPREADS = {"2^-13": np.where(np.arange(256) < 64, 2.0 ** -13, 1.0), "2^-14": np.where(np.arange(256) < 64, 2.0 ** -14, 1.0),
           "2^-16": np.where(np.arange(256) < 64, 2.0 ** -16, 1.0), "2^-20 to 1": 2.0 ** np.linspace(-20, 0, 256),
           "log-normal": np.exp(2 * np.random.default_rng(9).standard_normal(256))}


def longest_step(t, b1, b2):
    return (1 - b1) / (1 - b1 ** t) * np.sqrt((1 - b2 ** t) / (1 - b2) * sum((b1 * b1 / b2) ** k for k in range(t)))


@pytest.mark.parametrize("spread", SPREADS)
def test_steps_stay_as_long_as_exact_moments_allow(spread):
    r, b1, b2 = np.random.default_rng(0), 0.9, 0.999
    m, v = np.zeros(256), np.zeros(256)
    limit = 1.3 * max(longest_step(t, b1, b2) for t in (1, 2, 5, 10, 100, 1000))
    assert limit < 10
    for t in range(1, 1001):
        g = (r.standard_normal(256) * SPREADS[spread]).astype(np.float32)
        m, v = T.adamw_moments(m, v, g, b1, b2)
        u = T.adamw_weights(np.zeros(256), m.astype(float), v.astype(float), t, 1.0, b1, b2, 1e-8, 0.0)
        assert np.abs(u).max() <= limit, (t, np.abs(u).max())
        bits = r.integers(0, 65536, 256)
        m, _ = T.encode8(m, (bits & 255) << 8 | bits >> 8, 3, 7, 7)
        v, _ = T.encode8(v, bits, 2, 15, 14)


def test_a_second_moment_is_not_lost():
    """From its largest down to what is denormal in 32 bits it takes the smallest code at least; 0 and the first moments
    are as before."""
    x = np.zeros(256, dtype=np.float32)
    x[:5] = [2.0 ** 14, 2.0 ** -16, 2.0 ** -17, 1e-30, 1e-45]
    for r in (0, 65535):
        bits = np.full(256, r)
        q, s = T.encode8(x.view(T.SecondMoment), bits, 2, 15, 14)
        assert s[0] == 1 and q[0] == 2.0 ** 14 and (q[1:5] == 2.0 ** -16).all() and not q[5:].any()
        q, s = T.encode8(x, bits, 2, 15, 14)
        assert q[1] == 2.0 ** -16 and q[2] == (0 if r == 0 else 2.0 ** -16) and not q[3:].any()
