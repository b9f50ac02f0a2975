"""Pins of the training-pass oracle: published vectors of the generator,
closed forms, and every gradient against central differences in 64 bits."""

import numpy as np
import pytest

from oracle import train_ops as T


def test_philox_known_answers():
    """Random123's published Philox4x32-10 vectors."""
    cases = [((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
             ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
             ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
              (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]
    for c, k, want in cases:
        assert tuple(int(x) for x in T.philox4x32(np.array(c, dtype=np.uint64), k)) == want


def test_dropout_factor_keeps_the_mean():
    f = T.dropout_factor(400, 1003, 0.3, 7, 9)
    kept = (f > 0).mean()
    t = int(np.floor(65536 * np.float32(0.3) + 0.5))
    want = 1 - t / 65536
    assert abs(kept - want) < 5 * np.sqrt(want * (1 - want) / f.size)
    assert abs(f.max() * want - 1) < 1e-6


def differences(fn, x, h=1e-5):
    g = np.zeros_like(x)
    for at in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[at] += h
        b[at] -= h
        g[at] = (fn(a) - fn(b)) / (2 * h)
    return g


@pytest.mark.parametrize("nq,nk,causal,window", [(4, 4, False, 0), (5, 5, True, 0), (6, 4, True, 0), (3, 7, True, 2)])
def test_attention_gradient_is_the_difference_quotient(nq, nk, causal, window):
    r = np.random.default_rng(0)
    q, k, v, g = r.standard_normal((nq, 3)), r.standard_normal((nk, 3)), r.standard_normal((nk, 3)), r.standard_normal((nq, 3))
    see = T.visible(nq, nk, causal, window)
    got = T.attention(q, k, v, 0.7, see, g)
    f = lambda q, k, v: (T.attention(q, k, v, 0.7, see)["out"] * g).sum()  # noqa: E731
    assert np.allclose(got["dq"], differences(lambda x: f(x, k, v), q), atol=1e-8)
    assert np.allclose(got["dk"], differences(lambda x: f(q, x, v), k), atol=1e-8)
    assert np.allclose(got["dv"], differences(lambda x: f(q, k, x), v), atol=1e-8)
    empty = ~see.any(axis=1)
    assert empty.sum() == max(nq - nk, 0) * causal
    assert (got["out"][empty] == 0).all() and np.isneginf(got["lse"][empty]).all() and (got["dq"][empty] == 0).all()


def test_layer_norm_gradient_is_the_difference_quotient():
    r = np.random.default_rng(1)
    h, w, b, dy = r.standard_normal((3, 6)), r.standard_normal(6), r.standard_normal(6), r.standard_normal((3, 6))
    got = T.layer_norm_backward(dy, h, w, 1e-3)
    f = lambda h, w, b: (T.layer_norm(h, w, b, 1e-3)["y"] * dy).sum()  # noqa: E731
    assert np.allclose(got["g"], differences(lambda x: f(x, w, b), h), atol=1e-7)
    assert np.allclose(got["dweight"], differences(lambda x: f(h, x, b), w), atol=1e-7)
    assert np.allclose(got["dbias"], differences(lambda x: f(h, w, x), b), atol=1e-7)


@pytest.mark.parametrize("kl,scale", [(0.0, 1.0), (0.1, 0.5)])
def test_policy_gradient_is_the_difference_quotient(kl, scale):
    r = np.random.default_rng(2)
    x, t = r.standard_normal((6, 5)), np.array([0, 4, 2, 1, 1, 3])
    old = T.policy_loss(x, t, np.zeros(6), np.zeros(6), np.ones(6), np.ones(6), .2, .2, 0, scale)["logp"]
    old += np.array([0.5, -0.5, 0.1, -0.1, 0.3, 0.0])   # both sides of the clip, and inside it
    ref, adv, w = old + 0.2 * r.standard_normal(6), np.array([1, 1, -1, 1, -1, 2.0]), np.array([.2, .2, .2, .2, .2, 0])
    f = lambda x: T.policy_loss(x, t, old, ref, adv, w, .2, .25, kl, scale)["loss"]  # noqa: E731
    got = T.policy_loss(x, t, old, ref, adv, w, .2, .25, kl, scale)
    assert np.allclose(got["dlogits"], differences(f, x), atol=1e-8)
    assert (got["dlogits"][5] == 0).all()
