"""Cases for the training-pass operators: attention, layer norm, dropout and the
clipped policy loss, each with its backward pass.

``run`` computes a case either in its plain form (elementary torch operations in
32 bits, rounded once at the end) or, where ``own`` is true, through the calls of
``matrix_optimizer_step_02_amd.train``. ``exact`` states the same operators once
more in 64 bits.

Definitions that both forms share:

* Attention. Query i of a sequence sees key j where j < n_k, and with ``causal``
  j <= i + n_k - n_q, and with ``window`` w > 0 also j > i + n_k - n_q - w. A row
  that sees nothing has output 0, log-sum -inf and no gradient.
* Dropout. Element (r, c) of a rows x cols view takes 16 bits of Philox4x32-10
  (Salmon, Moraes, Dror, Shaw 2011): counter (c // 8, r, offset low, offset
  high), key (seed low, seed high), word (c % 8) // 2, its low half for even c.
  It is dropped where the 16 bits are below t = round(65536 p) and scaled by
  65536 / (65536 - t), rounded to 32 bits, otherwise.
* Layer norm. h = residual + dropout(x), product and sum each rounded to 32 bits
  and then to h's type, is an output of its own; y normalises that stored h.
* Policy loss. With logp the target's log probability under the logits,
  r = exp(logp - old), d = ref - logp:
  loss = sum_i w_i (max(-A r, -A clip(r, 1 - lo, 1 + hi)) + kl (exp(d) - d - 1)).
  Rows of weight 0 take no part: logp 0 and a gradient of zeros.
"""

import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # A chat-sized batch through one layer of a small model: launch latency.
        dict(name="attn fwd 4x128", op="attn", train=False, batch=4, q=128, k=128, heads=16, kv=16, dim=64,
             causal=True, window=0, dtype="bf16", ragged=False),
        # 509 new tokens scored against a context of 8192: few rows, a long key axis.
        dict(name="attn fwd 509 on 8192", op="attn", train=False, batch=1, q=509, k=8192, heads=16, kv=8, dim=128,
             causal=True, window=0, dtype="bf16", ragged=False),
        # One long document, grouped heads, the training pass (hidden 2048, k and v 1024 wide).
        dict(name="attn train 8192", op="attn", train=True, batch=1, q=8192, k=8192, heads=16, kv=8, dim=128,
             causal=True, window=0, dtype="bf16", ragged=False),
        # Documents of very different lengths packed into one batch of 8192 tokens.
        dict(name="attn train ragged", op="attn", train=True, batch=13, q=8192, k=8192, heads=16, kv=8, dim=128,
             causal=True, window=0, dtype="bf16", ragged=True),
        # Both directions visible, head width 64, float16, a length that ends inside a tile.
        dict(name="attn train 6x1000 f16", op="attn", train=True, batch=6, q=1000, k=1000, heads=16, kv=16, dim=64,
             causal=False, window=0, dtype="f16", ragged=False),
        # A norm over a few tokens: latency.
        dict(name="norm fwd 64x1024", op="norm", train=False, rows=64, cols=1024, dtype="bf16", res="bf16", p=0.0),
        # The norm of a layer of hidden 2048 over 16384 tokens, dropout and residual sum in the same pass.
        dict(name="norm train 16384x2048", op="norm", train=True, rows=16384, cols=2048, dtype="bf16", res="f32",
             p=0.1),
        # Odd sizes in 32 bits, no dropout.
        dict(name="norm train 4099x1000", op="norm", train=True, rows=4099, cols=1000, dtype="f32", res="f32",
             p=0.0),
        # Dropout alone: a small odd tensor, and the widest activation of a layer (FFN 6144).
        dict(name="dropout 1001x777", op="drop", rows=1001, cols=777, dtype="f32", res=False, p=0.25),
        dict(name="dropout 16384x6144", op="drop", rows=16384, cols=6144, dtype="bf16", res=True, p=0.1),
        # The loss of a short answer, and of a batch of 4096 tokens with a large vocabulary.
        dict(name="policy 61x32000", op="policy", rows=61, vocab=32000, dtype="f32", kl=0.04, lo=0.2, hi=0.2),
        dict(name="policy 4096x131072", op="policy", rows=4096, vocab=131072, dtype="bf16", kl=0.04, lo=0.2,
             hi=0.28),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "norm", "drop", "policy"])
    if op == "attn":
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4]) if kv < 8 else kv * rng.choice([1, 2])
        dim = rng.choice([64, 128, 128, 80, 96, 32])
        dtype = rng.choice(["bf16", "bf16", "f16"])
        causal = rng.random() < 0.7
        window = _log_int(rng, 16, 2048) if causal and rng.random() < 0.25 else 0
        train = rng.random() < 0.6
        if rng.random() < 0.4:
            total = _log_int(rng, 100, 8192)
            return dict(op="attn", train=train, batch=rng.randint(1, min(24, total // 4)), q=total, k=total,
                        heads=heads, kv=kv, dim=dim, causal=causal, window=window, dtype=dtype, ragged=True)
        q = _log_int(rng, 1, 6000)
        k = q if rng.random() < 0.7 else _log_int(rng, 1, 8192)
        batch = rng.randint(1, max(1, min(8, 6000 // max(q, k))))
        return dict(op="attn", train=train, batch=batch, q=q, k=k, heads=heads, kv=kv, dim=dim, causal=causal,
                    window=window, dtype=dtype, ragged=False)
    if op == "norm":
        cols = _log_int(rng, 16, 16384)
        rows = _log_int(rng, 1, max(1, min(32768, (1 << 25) // cols)))
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        return dict(op="norm", train=rng.random() < 0.7, rows=rows, cols=cols, dtype=dtype,
                    res=rng.choice(["none", "f32", dtype]), p=rng.choice([0.0, 0.0, 0.1, 0.3]))
    if op == "drop":
        cols = _log_int(rng, 1, 16384)
        rows = _log_int(rng, 1, max(1, min(32768, (1 << 26) // cols)))
        return dict(op="drop", rows=rows, cols=cols, dtype=rng.choice(["bf16", "f16", "f32"]),
                    res=rng.random() < 0.5, p=round(rng.uniform(0.02, 0.6), 3))
    vocab = _log_int(rng, 1000, 131072)
    rows = _log_int(rng, 1, max(1, min(8192, (1 << 28) // vocab)))
    return dict(op="policy", rows=rows, vocab=vocab, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                kl=rng.choice([0.0, 0.01, 0.1]), lo=0.2, hi=rng.choice([0.2, 0.28]))


def _lengths(case):
    """Sequence lengths of queries and keys. Ragged ones are packed: a heavy-tailed
    split of the total, of which one sequence has a single token."""
    b = case["batch"]
    if not case["ragged"]:
        return [case["q"]] * b, [case["k"]] * b
    r = random.Random(case["q"] * 131 + b)
    share = [math.exp(r.gauss(0.0, 1.0)) for _ in range(b)]
    room = case["q"] - b
    n = [1 + int(room * s / sum(share)) for s in share]
    if b > 2:
        n[-1] = 1
    n[0] += case["q"] - sum(n)
    return n, list(n)


def _pairs(case):
    total = 0
    for nq, nk in zip(*_lengths(case)):
        i = np.arange(nq, dtype=np.int64)
        hi = np.full(nq, nk, dtype=np.int64)
        lo = np.zeros(nq, dtype=np.int64)
        if case["causal"]:
            hi = np.clip(i + nk - nq + 1, 0, nk)
        if case["window"]:
            lo = np.clip(i + nk - nq - case["window"] + 1, 0, nk)
        total += int(np.maximum(hi - lo, 0).sum())
    return total


def work(case):
    op = case["op"]
    if op == "attn":
        e = _BYTES[case["dtype"]]
        nq, nk = (sum(x) for x in _lengths(case))
        q = nq * case["heads"] * case["dim"] * e
        kv = 2 * nk * case["kv"] * case["dim"] * e
        lse = nq * case["heads"] * 4
        f = 2.0 * _pairs(case) * case["heads"] * case["dim"]
        if case["train"]:   # also the output's gradient in, the gradients out
            return {"bytes": 4 * q + 2 * kv + lse, "flops": 7 * f}
        return {"bytes": 2 * q + kv + lse, "flops": 2 * f}
    n = case["rows"] * (case["vocab"] if op == "policy" else case["cols"])
    if op == "norm":
        e, r = _BYTES[case["dtype"]], _BYTES.get(case["res"], 0)
        he = r or e   # h is stored in the residual's type
        stored = bool(r) or case["p"] > 0
        b = n * (2 * e + r + (he if stored else 0)) + 8 * case["rows"] + 8 * case["cols"]
        f = 8.0 * n
        if case["train"]:   # dy and (with a residual) dh in; dx out, and the residual's gradient where it differs
            b += n * (e + r + e + (he if stored and (case["p"] > 0 or he != e) else 0)) + 8 * case["cols"]
            f += 14.0 * n
        return {"bytes": b, "flops": f}
    if op == "drop":
        return {"bytes": n * _BYTES[case["dtype"]] * (4 + (1 if case["res"] else 0)), "flops": 4.0 * n}
    return {"bytes": 2 * n * _BYTES[case["dtype"]] + 28 * case["rows"], "flops": 6.0 * n}


# ----------------------------------------------------------------- inputs ----

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(case)
    op = case["op"]
    dt = _DT[case["dtype"]]
    if op == "attn":
        b, h, kv, d = case["batch"], case["heads"], case["kv"], case["dim"]
        nq, nk = _lengths(case)
        s["scale"] = d ** -0.5
        s["max_q"], s["max_k"] = max(nq), max(nk)
        lead_q, lead_k = ((case["q"],), (case["k"],)) if case["ragged"] else ((b, case["q"]), (b, case["k"]))
        s["q_start"] = s["k_start"] = None
        if case["ragged"]:
            s["q_start"] = torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32, device=dev)
            s["k_start"] = torch.tensor(np.concatenate([[0], np.cumsum(nk)]), dtype=torch.int32, device=dev)
        if lead_q == lead_k:   # one projection's output: q, k and v are strided views of it
            qkv = randn(*lead_q, h + 2 * kv, d).to(dt)
            s["q"], s["k"], s["v"] = qkv.split([h, kv, kv], dim=-2)
        else:
            s["q"] = randn(*lead_q, h, d).to(dt)
            s["k"], s["v"] = randn(*lead_k, 2 * kv, d).to(dt).split([kv, kv], dim=-2)
        if case["train"]:
            s["dout"] = randn(*lead_q, h, d).to(dt)
    elif op == "norm":
        n, c = case["rows"], case["cols"]
        s["x"] = (1.5 * randn(n, c) + 0.25).to(dt)
        s["weight"], s["bias"] = 1 + 0.1 * randn(c), 0.1 * randn(c)
        s["residual"] = None if case["res"] == "none" else (2 * randn(n, c)).to(_DT[case["res"]])
        s["seed"], s["offset"] = seed * 7919 + 12345678901, seed + 3
        if case["train"]:
            s["dy"] = randn(n, c).to(dt)
            s["dh"] = None if s["residual"] is None else randn(n, c).to(_DT[case["res"]])
    elif op == "drop":
        n, c = case["rows"], case["cols"]
        s["x"] = randn(n, c).to(dt)
        s["residual"] = randn(n, c).to(dt) if case["res"] else None
        s["dy"] = randn(n, c).to(dt)
        s["seed"], s["offset"] = seed * 104729 + 98765432123, seed + 5
    else:
        n, v = case["rows"], case["vocab"]
        s["logits"] = randn(n, v).mul_(2.0).to(dt)
        s["target"] = torch.randint(0, v, (n,), generator=g, device=dev, dtype=torch.int32)
        rows = torch.arange(n, device=dev)
        s["logits"][rows, s["target"].long()] += 8.0   # a sampled token is a likely one
        lse = torch.cat([x.float().logsumexp(-1) for x in s["logits"].split(512)])
        logp = s["logits"][rows, s["target"].long()].float() - lse
        gap = 0.25 * randn(n)
        # no row within rounding of the clip's borders, where either branch is right
        for edge in (math.log(1 - case["lo"]), math.log(1 + case["hi"])):
            gap = torch.where((gap - edge).abs() < 1e-2, gap + 3e-2, gap)
        s["old_logp"] = logp - gap
        s["ref_logp"] = logp + 0.3 * randn(n)
        s["advantage"] = randn(n) + 0.1
        keep = (torch.rand(n, generator=g, device=dev) < 0.8).float()   # prompts and padding have weight 0
        keep[0] = 1.0
        s["weight"] = keep / keep.sum()
    return s


# ------------------------------------------------------------ plain forms ----

def _pad(x, start, most):
    """Packed rows (N, heads, dim) as (batch, most, heads, dim) and each slot's row (N where there is none)."""
    n = x.shape[0]
    t = torch.arange(most, device=x.device)
    row = start[:-1, None].long() + t
    row = torch.where(row < start[1:, None].long(), row, n)
    return x[row.clamp(max=n - 1)], row


def _unpad(x, row, n):
    """(batch, most, ...) back to n packed rows; slots without a row go to one that is cut off."""
    out = torch.empty(n + 1, *x.shape[2:], dtype=x.dtype, device=x.device)
    out[row.reshape(-1)] = x.reshape(-1, *x.shape[2:])
    return out[:n]


def _plain_attention(s):
    q, k, v = (s[n].float() for n in "qkv")
    dev, dt = q.device, s["q"].dtype
    rq = rk = None
    if s["ragged"]:
        n = q.shape[0]
        q, rq = _pad(q, s["q_start"], s["max_q"])
        k, rk = _pad(k, s["k_start"], s["max_k"])
        v, _ = _pad(v, s["k_start"], s["max_k"])
        lq = (s["q_start"][1:] - s["q_start"][:-1]).long().view(-1, 1, 1)
        lk = (s["k_start"][1:] - s["k_start"][:-1]).long().view(-1, 1, 1)
    else:
        lq = torch.full((1, 1, 1), s["q"].shape[1], device=dev)
        lk = torch.full((1, 1, 1), s["k"].shape[1], device=dev)
    group = s["heads"] // s["kv"]
    q = q.transpose(1, 2).contiguous()
    k, v = (x.transpose(1, 2).repeat_interleave(group, dim=1) for x in (k, v))
    i = torch.arange(q.shape[2], device=dev).view(1, -1, 1)
    j = torch.arange(k.shape[2], device=dev).view(1, 1, -1)
    see = (j < lk) & (i < lq)
    if s["causal"]:
        see = see & (j <= i + lk - lq)
    if s["window"]:
        see = see & (j > i + lk - lq - s["window"])
    see = see.unsqueeze(1)
    p = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(s["scale"])
    p = p.masked_fill_(~see, -math.inf)
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    p = p.div_(torch.where(total > 0, total, 1.0))
    out = torch.matmul(p, v)

    def back(x, row):
        x = x.transpose(1, 2)
        return (x if row is None else _unpad(x, row, n)).to(dt)

    def lse_back(x):
        if rq is None:
            return x.transpose(0, 1).reshape(x.shape[1], -1)
        return _unpad(x.transpose(1, 2), rq, n).t().contiguous()

    if not s["train"]:
        return {"out": back(out, rq), "lse": lse_back(lse)}
    do = s["dout"].float()
    if s["ragged"]:
        do, _ = _pad(do, s["q_start"], s["max_q"])
    do = do.transpose(1, 2).contiguous()
    dv = torch.matmul(p.transpose(-1, -2), do)
    dp = torch.matmul(do, v.transpose(-1, -2).contiguous())
    ds = dp.sub_((dp * p).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q)
    dk, dv = (x.reshape(x.shape[0], s["kv"], group, *x.shape[2:]).sum(2) for x in (dk, dv))
    return {"out": back(out, rq), "lse": lse_back(lse), "dq": back(dq, rq), "dk": back(dk, rk), "dv": back(dv, rk)}


def _keep(rows, cols, p, seed, offset, dev):
    """(rows, cols) truth values: what dropout keeps. 64-bit integers, products modulo 2^64."""
    low = 0xFFFFFFFF
    groups = (cols + 7) // 8
    c0 = torch.arange(groups, device=dev).expand(rows, groups)
    c1 = torch.arange(rows, device=dev).view(-1, 1).expand(rows, groups)
    c2, c3 = torch.full_like(c0, offset & low), torch.full_like(c0, offset >> 32 & low)
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & low) ^ c1 ^ k0, b & low, (a >> 32 & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((c0, c1, c2, c3), -1)
    bits = torch.stack((words & 0xFFFF, words >> 16), -1).reshape(rows, groups * 8)[:, :cols]
    return bits >= _threshold(p)


def _threshold(p):
    return int(round(65536 * p))


def _plain_dropout(x, s):
    if s["p"] == 0:
        return x.float()
    t = _threshold(s["p"])
    scale = float(np.float32(65536.0 / (65536 - t)))
    keep = _keep(x.shape[0], x.shape[1], s["p"], s["seed"], s["offset"], x.device)
    return torch.where(keep, x.float() * scale, 0.0)


def _plain_norm(s):
    x, res = s["x"], s["residual"]
    h = _plain_dropout(x, s)
    ht = x.dtype if res is None else res.dtype
    h = (h if res is None else res.float() + h).to(ht)
    f = h.float()
    mean = f.mean(-1)
    d = f - mean[:, None]
    rstd = (d.square().mean(-1) + 1e-5).rsqrt()
    xhat = d * rstd[:, None]
    out = {"y": (xhat * s["weight"] + s["bias"]).to(x.dtype), "h": h, "mean": mean, "rstd": rstd}
    if s["train"]:
        dy = s["dy"].float()
        wd = dy * s["weight"]
        dh = (wd - wd.mean(-1, keepdim=True) - xhat * (wd * xhat).mean(-1, keepdim=True)) * rstd[:, None]
        if s["dh"] is not None:
            dh = dh + s["dh"].float()
        out["dx"] = _plain_dropout(dh, s).to(x.dtype)
        if res is not None:
            out["dres"] = dh.to(ht)
        out["dweight"], out["dbias"] = (dy * xhat).sum(0), dy.sum(0)
    return out


def _plain_drop(s):
    y = _plain_dropout(s["x"], s)
    if s["residual"] is not None:
        y = s["residual"].float() + y
    return {"y": y.to(s["x"].dtype), "dx": _plain_dropout(s["dy"], s).to(s["x"].dtype)}


def _plain_policy(s):
    z = s["logits"].float()
    w = s["weight"]
    at = s["target"].long()[:, None]
    top = z.amax(-1, keepdim=True)
    e = (z - top).exp_()
    total = e.sum(-1, keepdim=True)
    logp = (z.gather(1, at) - top - total.log()).squeeze(1)
    used = w != 0
    r = (logp - s["old_logp"]).exp()
    a = s["advantage"]
    free, clipped = -a * r, -a * r.clamp(1 - s["lo"], 1 + s["hi"])
    d = s["ref_logp"] - logp
    term = torch.maximum(free, clipped) + s["kl"] * (d.exp() - d - 1)
    loss = torch.where(used, w * term, 0.0).sum()
    slope = torch.where(free >= clipped, free, 0.0) + s["kl"] * (1 - d.exp())
    slope = torch.where(used, w * slope, 0.0)
    grad = e.mul_(-slope[:, None] / total)
    grad.scatter_add_(1, at, slope[:, None])
    return {"loss": loss, "logp": torch.where(used, logp, 0.0), "dlogits": grad.to(s["logits"].dtype)}


# ----------------------------------------------------------------- passes ----

def run(s):
    op = s["op"]
    if not own:
        return {"attn": _plain_attention, "norm": _plain_norm, "drop": _plain_drop, "policy": _plain_policy}[op](s)
    from matrix_optimizer_step_02_amd import train
    if op == "attn":
        how = dict(causal=s["causal"], window=s["window"], scale=s["scale"], q_start=s["q_start"],
                   k_start=s["k_start"], max_q=s["max_q"], max_k=s["max_k"])
        out, lse = train.attention_forward(s["q"], s["k"], s["v"], **how)
        if not s["train"]:
            return {"out": out, "lse": lse}
        dq, dk, dv = train.attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, **how)
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if op == "norm":
        rng = train.Rng(s["seed"], s["offset"])
        y, h, mean, rstd = train.layer_norm_forward(s["x"], s["weight"], s["bias"], eps=1e-5,
                                                    residual=s["residual"], p=s["p"], rng=rng)
        out = {"y": y, "h": h, "mean": mean, "rstd": rstd}
        if s["train"]:
            res = s["residual"] is not None
            dx, dres, out["dweight"], out["dbias"] = train.layer_norm_backward(
                s["dy"], h, s["weight"], mean, rstd, dh=s["dh"], p=s["p"], rng=rng, residual_grad=res)
            out |= {"dx": dx, "dres": dres} if res else {"dx": dx}
        return out
    if op == "drop":
        rng = train.Rng(s["seed"], s["offset"])
        return {"y": train.dropout(s["x"], s["p"], rng, residual=s["residual"]),
                "dx": train.dropout_backward(s["dy"], s["p"], rng)}
    loss, logp, dlogits = train.policy_loss_step(
        s["logits"], s["target"], s["old_logp"], s["advantage"], s["weight"], ref_logp=s["ref_logp"],
        clip_low=s["lo"], clip_high=s["hi"], kl_coef=s["kl"])
    return {"loss": loss, "logp": logp, "dlogits": dlogits}


# ---------------------------------------------------------------- 64 bits ----

def _exact_attention(case, s):
    q, k, v = (s[n].double() for n in "qkv")
    do = s["dout"].double() if case["train"] else None
    nq, nk = _lengths(case)
    group = case["heads"] // case["kv"]
    flat_q = q.reshape(-1, case["heads"], case["dim"])
    flat_k, flat_v = (x.reshape(-1, case["kv"], case["dim"]) for x in (k, v))
    out, dq = torch.zeros_like(flat_q), torch.zeros_like(flat_q)
    dk, dv = torch.zeros_like(flat_k), torch.zeros_like(flat_v)
    lse = torch.full((case["heads"], flat_q.shape[0]), -math.inf, dtype=torch.float64, device=q.device)
    if do is not None:
        do = do.reshape(flat_q.shape)
    a = c = 0
    for m, n in zip(nq, nk):
        last = torch.arange(m, device=q.device)[:, None] + (n - m) if case["causal"] else torch.full(
            (m, 1), n - 1, device=q.device)
        key = torch.arange(n, device=q.device)[None]
        hide = key > last
        if case["window"]:
            hide |= key <= torch.arange(m, device=q.device)[:, None] + (n - m) - case["window"]
        for h in range(case["heads"]):
            qs, ks, vs = flat_q[a:a + m, h], flat_k[c:c + n, h // group], flat_v[c:c + n, h // group]
            sc = torch.where(hide, -math.inf, qs @ ks.t().contiguous() * s["scale"])
            z = torch.logsumexp(sc, 1)
            lse[h, a:a + m] = z
            p = torch.where(hide, 0.0, (sc - torch.where(z.isinf(), 0.0, z)[:, None]).exp())
            o = p @ vs
            out[a:a + m, h] = o
            if do is not None:
                g = do[a:a + m, h]
                ds = p * (g @ vs.t().contiguous() - (g * o).sum(1, keepdim=True)) * s["scale"]
                dq[a:a + m, h] = ds @ ks
                dk[c:c + n, h // group] += ds.t().contiguous() @ qs
                dv[c:c + n, h // group] += p.t().contiguous() @ g
        a, c = a + m, c + n
    got = {"out": out.view(q.shape), "lse": lse}
    if do is not None:
        got |= {"dq": dq.view(q.shape), "dk": dk.view(k.shape), "dv": dv.view(v.shape)}
    return got


def _exact_drop(x, s, ties32=False):
    """x in 64 bits through dropout; ``ties32``: the product rounded to 32 bits, as the operator defines h."""
    t = int(round(65536 * s["p"]))
    if not t:
        return x
    scale = np.float32(65536.0 / (65536 - t)).item()
    words = _philox(x.shape[0], (x.shape[1] + 7) // 8, s["seed"], s["offset"])
    bits = torch.from_numpy(words.view("<u2").astype(np.int32)).to(x.device)
    keep = bits.view(x.shape[0], -1)[:, :x.shape[1]] >= t
    y = x * scale
    return torch.where(keep, y.float().double() if ties32 else y, 0.0)


def _philox(rows, groups, seed, offset):
    """(rows, groups, 4) 32-bit words."""
    u = np.uint64
    low, half = u(0xFFFFFFFF), u(32)
    got = np.empty((rows, groups, 4), dtype="<u4")
    step = max(1, (1 << 22) // groups)
    for r in range(0, rows, step):
        e = min(rows, r + step)
        x = [np.tile(np.arange(groups, dtype=u), (e - r, 1)), np.repeat(np.arange(r, e, dtype=u)[:, None], groups, 1),
             np.full((e - r, groups), offset & 0xFFFFFFFF, dtype=u), np.full((e - r, groups), offset >> 32, dtype=u)]
        for n in range(10):
            key = [u((seed + n * 0x9E3779B9) & 0xFFFFFFFF), u(((seed >> 32) + n * 0xBB67AE85) & 0xFFFFFFFF)]
            p0, p1 = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
            x = [(p1 >> half) ^ x[1] ^ key[0], p1 & low, (p0 >> half) ^ x[3] ^ key[1], p0 & low]
        for w in range(4):
            got[r:e, :, w] = x[w]
    return got


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attn":
        return _exact_attention(case, s)
    if op == "drop":
        y = _exact_drop(s["x"].double(), s)
        return {"y": y if s["residual"] is None else y + s["residual"].double(),
                "dx": _exact_drop(s["dy"].double(), s)}
    if op == "norm":
        h = _exact_drop(s["x"].double(), s, ties32=True)
        if s["residual"] is not None:
            h = (h + s["residual"].double()).float()
        h = h.to(s["x"].dtype if s["residual"] is None else s["residual"].dtype).double()
        w, b = s["weight"].double(), s["bias"].double()
        var, mean = torch.var_mean(h, 1, correction=0, keepdim=True)
        rstd = 1 / torch.sqrt(var + 1e-5)
        z = (h - mean) * rstd
        got = {"y": z * w + b, "h": h, "mean": mean[:, 0], "rstd": rstd[:, 0]}
        if case["train"]:
            dy = s["dy"].double()
            dz = dy * w
            dh = rstd * (dz - dz.mean(1, keepdim=True) - z * (dz * z).mean(1, keepdim=True))
            if s["dh"] is not None:
                dh += s["dh"].double()
            got |= {"dx": _exact_drop(dh, s), "dweight": (dy * z).sum(0), "dbias": dy.sum(0)}
            if s["residual"] is not None:
                got["dres"] = dh
        return got
    n = case["rows"]
    rows = torch.arange(n, device=s["logits"].device)
    t = s["target"].long()
    w, old, ref, adv = (s[x].double() for x in ("weight", "old_logp", "ref_logp", "advantage"))
    grad = torch.empty(s["logits"].shape, dtype=torch.float64, device=rows.device)
    logp = torch.empty(n, dtype=torch.float64, device=rows.device)
    for at in rows.split(256):
        z = torch.log_softmax(s["logits"][at].double(), -1)
        logp[at] = z.gather(1, t[at][:, None])[:, 0]
        grad[at] = -z.exp()
    grad[rows, t] += 1
    ratio = torch.exp(logp - old)
    bounded = ratio.clip(1 - case["lo"], 1 + case["hi"])
    gain = torch.minimum(adv * ratio, adv * bounded)
    kl = torch.expm1(ref - logp) - (ref - logp)
    slope = -adv * ratio * (adv * ratio <= adv * bounded) - case["kl"] * torch.expm1(ref - logp)
    live = (w != 0).double()
    grad *= (w * slope)[:, None]
    return {"loss": (w * (case["kl"] * kl - gain)).sum(), "logp": logp * live, "dlogits": grad}
