"""fp64 oracle of the training-pass operators (attention, layer norm, dropout,
clipped policy loss) and their gradients, from the formulas; numpy only."""

from __future__ import annotations

import numpy as np


# -------------------------------------------------------------- attention ----


def visible(nq, nk, causal=False, window=0, sinks=0):
    """(nq, nk) truth values: key j < nk, j <= i + nk - nq, j > i + nk - nq - window or j < sinks."""
    i, j = np.arange(nq)[:, None] + nk - nq, np.arange(nk)[None]
    see = np.ones((nq, nk), dtype=bool)
    if causal:
        see &= j <= i
    if window:
        see &= (j > i - window) | (j < sinks)
    return see


def attention(q, k, v, scale, see, dout=None):
    """One head: q (nq, d), k and v (nk, d). Returns a dict with out, lse, p
    and, with dout, dq, dk, dv, dp, D, ds."""
    s = np.where(see, scale * (q @ k.T), -np.inf)
    top = np.max(s, axis=1, initial=-np.inf)
    top0 = np.where(np.isfinite(top), top, 0.0)
    e = np.where(see, np.exp(s - top0[:, None]), 0.0)
    total = e.sum(axis=1)
    with np.errstate(divide="ignore"):
        lse = top0 + np.log(total)
    p = e / np.where(total > 0, total, 1.0)[:, None]
    r = {"out": p @ v, "lse": lse, "p": p}
    if dout is not None:
        dp = dout @ v.T
        D = (dout * r["out"]).sum(axis=1)
        ds = p * (dp - D[:, None])
        r |= {"dp": dp, "D": D, "ds": ds, "dq": scale * ds @ k, "dk": scale * ds.T @ q, "dv": p.T @ dout}
    return r


# ---------------------------------------------------------------- dropout ----


def philox4x32(counter, key, rounds=10):
    """Philox4x32 of (..., 4) counters and a (k0, k1) key."""
    x = [np.asarray(counter[..., n], dtype=np.uint64) for n in range(4)]
    k = [np.uint64(key[0]), np.uint64(key[1])]
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> half) ^ x[1] ^ k[0], b & low, (a >> half) ^ x[3] ^ k[1], a & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return np.stack(x, axis=-1).astype(np.uint32)


def dropout_factor(rows, cols, p, seed, offset):
    """(rows, cols) float32 factors: 0, or 65536 / (65536 - round(65536 p))."""
    t = int(np.floor(65536 * float(np.float32(p)) + 0.5))
    groups = (cols + 7) // 8
    c = np.zeros((rows, groups, 4), dtype=np.uint64)
    c[..., 0], c[..., 1] = np.arange(groups)[None], np.arange(rows)[:, None]
    c[..., 2], c[..., 3] = offset & 0xFFFFFFFF, (offset >> 32) & 0xFFFFFFFF
    w = philox4x32(c, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    bits = np.stack([w & 0xFFFF, w >> 16], axis=-1).reshape(rows, groups * 8)[:, :cols]
    return np.where(bits >= t, np.float32(65536.0 / (65536 - t)), np.float32(0))


# ------------------------------------------------------------- layer norm ----


def layer_norm(h, w, b, eps):
    mean = h.mean(axis=1)
    rstd = 1 / np.sqrt(((h - mean[:, None]) ** 2).mean(axis=1) + eps)
    xh = (h - mean[:, None]) * rstd[:, None]
    return {"y": xh * w + (0 if b is None else b), "mean": mean, "rstd": rstd, "xh": xh}


def layer_norm_backward(dy, h, w, eps, dh=None):
    f = layer_norm(h, w, None, eps)
    xh, z = f["xh"], dy * w
    g = f["rstd"][:, None] * (z - z.mean(1, keepdims=True) - xh * (z * xh).mean(1, keepdims=True))
    if dh is not None:
        g = g + dh
    return {"g": g, "dweight": (dy * xh).sum(0), "dbias": dy.sum(0), "xh": xh, "z": z, "rstd": f["rstd"]}


# ------------------------------------------------------------ policy loss ----


def policy_loss(x, target, old, ref, adv, w, lo, hi, kl, scale=1.0, grad=1.0):
    """Rows of weight 0 contribute nothing, whatever they hold."""
    n, v = x.shape
    logp, lse, slope, term = (np.zeros(n) for _ in range(4))
    dx = np.zeros((n, v))
    for i in range(n):
        if w[i] == 0:
            continue
        z = scale * x[i]
        m = z.max()
        lse[i] = m + np.log(np.exp(z - m).sum())
        if not 0 <= target[i] < v:
            logp[i] = slope[i] = term[i] = np.nan
            dx[i] = np.nan
            continue
        logp[i] = z[target[i]] - lse[i]
        r = np.exp(logp[i] - old[i])
        free, bound = -adv[i] * r, -adv[i] * min(max(r, 1 - lo), 1 + hi)
        term[i], slope[i] = max(free, bound), free if free >= bound else 0.0
        if kl:
            d = ref[i] - logp[i]
            term[i] += kl * (np.expm1(d) - d)
            slope[i] -= kl * np.expm1(d)
        term[i] *= w[i]
        slope[i] *= w[i]
        dx[i] = -np.exp(z - lse[i])
        dx[i, target[i]] += 1
        dx[i] *= grad * scale * slope[i]
    return {"loss": term.sum(), "logp": logp, "lse": lse, "slope": slope, "dlogits": dx, "term": term}


# --------------------------------------------------- rotary and qk norm ----


def rotary(x, positions, frequencies, layout="half", scale=1.0, inverse=False):
    """x (tokens, heads, dim), positions (tokens,) integers. Angles from exact integer positions: the product with a
    frequency is reduced by whole turns in extended precision."""
    turns = np.asarray(positions, dtype=np.longdouble)[:, None] * (
        np.asarray(frequencies, dtype=np.longdouble) / (2 * np.longdouble("3.14159265358979323846264338327950288")))
    angle = ((turns - np.round(turns)) * 2).astype(np.float64)[:, None] * np.pi
    c, s = scale * np.cos(angle), scale * np.sin(angle) * (-1 if inverse else 1)
    rot, y = 2 * len(frequencies), x.copy()
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def rms_norm(x, w, eps):
    """Rows along the last axis: y, rstd, xh."""
    rstd = 1 / np.sqrt((x ** 2).mean(-1) + eps)
    xh = x * rstd[..., None]
    return {"y": xh * w, "rstd": rstd, "xh": xh}


def rms_norm_backward(g, x, w, eps):
    f = rms_norm(x, w, eps)
    z, xh = g * w, f["xh"]
    dx = f["rstd"][..., None] * (z - xh * (z * xh).mean(-1, keepdims=True))
    return {"dx": dx, "dw": (g * xh).reshape(-1, x.shape[-1]).sum(0), "z": z} | f


# ------------------------------------------------------------------ AdamW ----


class SecondMoment(np.ndarray):
    """Averages of squares, of which encode8 makes no 0 that was none."""


def adamw_moments(m, v, g, b1, b2):
    """In float32, each product and sum rounded: what the states of 8 bits are made from."""
    f = np.float32
    m, v, g = (np.asarray(x, dtype=f) for x in (m, v, g))
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        return m * f(b1) + g * f(1 - b1), (v * f(b2) + (g * g) * f(1 - b2)).view(SecondMoment)


def adamw_weights(w, m, v, t, lr, b1, b2, eps, decay):
    """In float64, from the moments after step t."""
    u = m / (1 - b1 ** t) / (np.sqrt(np.asarray(v) / (1 - b2 ** t)) + eps)
    return w - lr * (u + decay * w)


def random16(n, tensor, seed, offset, first=0):
    """The 16 random bits of n elements of a tensor from element ``first``, a multiple of 8, on."""
    groups = (n + 7) // 8
    c = np.zeros((groups, 4), dtype=np.uint64)
    c[:, 0], c[:, 1], c[:, 2], c[:, 3] = first // 8 + np.arange(groups), tensor, offset & 0xFFFFFFFF, (offset >> 32) & 0xFFFFFFFF
    w = philox4x32(c, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    return np.stack([w & 0xFFFF, w >> 16], axis=-1).reshape(-1)[:n].astype(np.int64)


def encode8(x, r, digits, bias, top, block=256):
    """(values, scales): x (float32) in blocks with a power of two each, rounded up in magnitude where the discarded
    fraction plus r / 65536 reaches 1, and a second moment that is not 0 to the smallest code at least. Values are what
    the codes stand for, scale included; NaN where x is not finite."""
    second, x = isinstance(x, SecondMoment), np.asarray(x)
    n, f = x.size, np.float64
    mag = np.abs(np.pad(x.astype(f), (0, -n % block)).reshape(-1, block))
    big = np.where(np.isfinite(mag), mag, 0).max(axis=1)
    _, e = np.frexp(big)   # big = f 2^e, f in [1/2, 1)
    e = np.clip(np.where(big > 0, e - 1 - top, -200), -120, 120)
    scale = np.ldexp(1.0, e)
    with np.errstate(invalid="ignore"):
        y = (mag / scale[:, None]).reshape(-1)[:n]
        _, ye = np.frexp(np.where(np.isfinite(y), y, 1.0))
        step = np.ldexp(1.0, np.maximum(ye - 1, 1 - bias) - digits)
        q = np.floor(y / step + r / 65536) * step
        if second:
            q = np.where((y > 0) & (q == 0), step, q)
    q = np.where(np.isfinite(x), np.copysign(q, x), np.nan)
    return q * np.repeat(scale, block)[:n], scale
