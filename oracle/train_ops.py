"""fp64 oracle of the training-pass operators (attention, layer norm, dropout,
clipped policy loss) and their gradients, from the formulas; numpy only."""

from __future__ import annotations

import numpy as np


# -------------------------------------------------------------- attention ----


def visible(nq, nk, causal=False, window=0):
    """(nq, nk) truth values: key j < nk, j <= i + nk - nq, j > i + nk - nq - window."""
    i, j = np.arange(nq)[:, None] + nk - nq, np.arange(nk)[None]
    see = np.ones((nq, nk), dtype=bool)
    if causal:
        see &= j <= i
    if window:
        see &= j > i - window
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
