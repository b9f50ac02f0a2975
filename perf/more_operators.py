"""Cases for position rotation, norms of queries and keys with the rotation, attention
with a sliding window and first tokens that stay visible (sinks), and the AdamW step
over many tensors with states in 32 or 8 bits.

``run`` computes a case either in its plain form (elementary torch operations in
32 bits, angles in 64, rounded once at the end) or, where ``own`` is true, through the
framework's calls. ``exact`` states the same operators once more in 64 bits.

Definitions that both forms share:

* Rotation. Pair i of a head at position p turns by the angle p f_i:
  (a, b) -> s (a cos - b sin, b cos + a sin). Layout "half" pairs element i with
  i + rot / 2, "pairs" 2 i with 2 i + 1; elements from rot on stay. The gradient
  turns back. Frequencies: f_i = base^(-2 i / rot); "linear" divides them by a
  factor, "base" raises the base to base factor^(rot / (rot - 2)), "ramp" divides
  those that turn fewer than 1 times over the original length, keeps those that
  turn more than 32 times, goes linearly between, and scales by s = 1 + 0.1 ln factor
  (Peng, Quesnel, Fan, Shippole 2023).
* Norm per head. y = rotation(x rstd w), rstd = 1 / sqrt(mean(x^2) + eps) over a
  head's elements.
* Attention. Query i sees key j where j <= i + n_k - n_q and (j > i + n_k - n_q -
  window or j < sinks).
* AdamW, step t, gradient g = scale G: m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2
  (each product and sum rounded to 32 bits),
  W = W - lr (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + decay W).
  States in 8 bits: blocks of 256 elements of a tensor, m as e4m3 and v as e5m2 times
  a power of two that puts the block's largest magnitude into [2^7, 2^8) or
  [2^14, 2^15), rounded up where the discarded fraction plus r / 65536 reaches 1.
  r are 16 bits of Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011): element i of
  tensor n takes counter (i // 8, n, offset low, offset high), key (seed low, seed
  high), word (i % 8) // 2, its low half for even i; m takes them with the two bytes
  exchanged.
"""

import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
_BLOCK = 256
_ADAM = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # One new token of each of 16 conversations, at positions far apart: launch latency.
        dict(name="rotary 16 new tokens", op="rotary", train=False, batch=16, tokens=1, heads=16, kv=8, dim=128,
             rot=128, layout="half", scaling="none", factor=1.0, at="list", far=32768, dtype="bf16"),
        # Queries and keys of a layer of hidden 2048 over 16384 tokens of packed documents, forward and backward.
        dict(name="rotary train 16384", op="rotary", train=True, batch=1, tokens=16384, heads=16, kv=8, dim=128,
             rot=128, layout="half", scaling="ramp", factor=4.0, at="list", far=131072, dtype="bf16"),
        # Odd sizes, part of the head, neighbouring pairs, 32 bits, positions of a long file.
        dict(name="rotary train 3x1021 f32", op="rotary", train=True, batch=3, tokens=1021, heads=7, kv=7, dim=80,
             rot=44, layout="pairs", scaling="linear", factor=8.0, at="ramp", far=1 << 20, dtype="f32"),
        # The same new tokens with norms of queries and keys before the rotation.
        dict(name="qk norm 16 new tokens", op="norm", train=False, batch=16, tokens=1, heads=16, kv=8, dim=128,
             rot=128, layout="half", scaling="none", factor=1.0, at="list", far=32768, dtype="bf16"),
        # A layer of hidden 2048 over 16384 tokens, with the gradients of queries, keys and both weights.
        dict(name="qk norm train 16384", op="norm", train=True, batch=2, tokens=8192, heads=16, kv=8, dim=128,
             rot=128, layout="half", scaling="none", factor=1.0, at="ramp", far=0, dtype="bf16"),
        # Narrow heads in float16, part of the head turned, more query heads to a key head, odd lengths.
        dict(name="qk norm train 5x999 f16", op="norm", train=True, batch=5, tokens=999, heads=12, kv=3, dim=72,
             rot=36, layout="pairs", scaling="base", factor=2.0, at="list", far=50000, dtype="f16"),
        # One new token of each of 32 conversations on up to 8192 keys: bytes of the keys and values in sight.
        dict(name="sinks fwd 32x1 on 8192", op="attn", train=False, batch=32, q=1, k=8192, heads=16, kv=8, dim=128,
             window=4096, sinks=4, dtype="bf16", lengths="padded"),
        # One long document with a window, the training pass.
        dict(name="sinks train 8192", op="attn", train=True, batch=1, q=8192, k=8192, heads=16, kv=8, dim=128,
             window=1024, sinks=4, dtype="bf16", lengths="full"),
        # Packed documents of very different lengths, narrow heads, a window and sinks that end inside tiles.
        dict(name="sinks train ragged f16", op="attn", train=True, batch=9, q=6007, k=6007, heads=16, kv=4, dim=64,
             window=200, sinks=37, dtype="f16", lengths="packed"),
        # Norm weights and biases of a model of 28 layers: latency of many small tensors.
        dict(name="adamw 142 small", op="adamw", bits=32, count=142, total=172800, largest=2048, grad="f32", copy="none",
             clip=False),
        # An embedding of 65536 tokens, hidden 2048, and what else is no matrix: bf16 gradients, clipping, bf16 copy.
        dict(name="adamw embedding 32 bit", op="adamw", bits=32, count=60, total=134300000, largest=134217728,
             grad="bf16", copy="bf16", clip=True),
        # The same with states in 8 bits and 32-bit gradients.
        dict(name="adamw embedding 8 bit", op="adamw", bits=8, count=60, total=134300001, largest=134217728, grad="f32",
             copy="bf16", clip=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "norm", "norm", "attn", "attn", "attn", "adamw", "adamw"])
    if op in ("rotary", "norm"):
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 2, 4])
        dim = rng.choice([32, 64, 64, 72, 80, 96, 128, 128, 128, 160, 256])
        rot = dim if rng.random() < 0.6 else 2 * rng.randint(2, dim // 2)
        tokens = _log_int(rng, 1, max(1, min(16384, (1 << 25) // ((heads + kv) * dim))))
        batch = rng.randint(1, max(1, min(16, 16384 // tokens, (1 << 25) // (tokens * (heads + kv) * dim))))
        scaling = rng.choice(["none", "none", "linear", "base", "ramp"])
        return dict(op=op, train=rng.random() < 0.7, batch=batch, tokens=tokens, heads=heads, kv=kv, dim=dim, rot=rot,
                    layout=rng.choice(["half", "pairs"]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]), at=rng.choice(["ramp", "list"]),
                    far=_log_int(rng, 64, 1 << 20), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op == "attn":
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4]) if kv < 8 else kv * rng.choice([1, 2])
        dim = rng.choice([64, 128, 128, 80, 96, 32])
        window, sinks = _log_int(rng, 1, 2048), rng.choice([1, 4, 4, 16, 37, 64, 130])
        dtype = rng.choice(["bf16", "bf16", "f16"])
        train = rng.random() < 0.6
        lengths = rng.choice(["full", "packed", "padded"])
        if lengths == "packed":
            total = _log_int(rng, 100, 8000)
            return dict(op="attn", train=train, batch=rng.randint(1, min(24, total // 4)), q=total, k=total,
                        heads=heads, kv=kv, dim=dim, window=window, sinks=sinks, dtype=dtype, lengths=lengths)
        k = _log_int(rng, 1, 8000)
        q = rng.choice([1, k, k, _log_int(rng, 1, 2000)])
        batch = rng.randint(1, max(1, min(24, 12000 // max(q, k))))
        return dict(op="attn", train=train, batch=batch, q=q, k=k, heads=heads, kv=kv, dim=dim, window=window,
                    sinks=sinks, dtype=dtype, lengths=lengths)
    count = _log_int(rng, 1, 200)
    largest = _log_int(rng, 1, 1 << 25)
    return dict(op="adamw", bits=rng.choice([32, 32, 8, 8]), count=count,
                total=largest + (count - 1) * _log_int(rng, 1, min(largest, 1 << 17)), largest=largest,
                grad=rng.choice(["bf16", "f16", "f32"]), copy=rng.choice(["none", "bf16", "f16"]),
                clip=rng.random() < 0.4)


def _lengths(case):
    """Tokens of each sequence's queries and keys. Packed: a heavy-tailed split of the total, one sequence of a
    single token. Padded: keys from a few to all, of which the queries are the last."""
    b = case["batch"]
    if case["lengths"] == "full":
        return [case["q"]] * b, [case["k"]] * b
    r = random.Random(case["q"] * 131 + case["k"] * 7 + b)
    if case["lengths"] == "padded":
        nk = [r.randint(1 + case["k"] // 3, case["k"]) if case["k"] > 2 else case["k"] for _ in range(b)]
        nk[0] = case["k"]
        return [min(case["q"], n) for n in nk], nk
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
        hi = np.clip(np.arange(nq, dtype=np.int64) + nk - nq + 1, 0, nk)
        lo = np.clip(hi - case["window"], 0, nk)
        total += int((hi - lo + np.minimum(lo, case["sinks"])).sum())
    return total


def _sizes(case):
    """Elements of each tensor: the largest, single ones, and the rest between."""
    n, rest = case["count"] - 1, case["total"] - case["largest"]
    if n == 0:
        return [case["largest"]]
    r = random.Random(case["count"] * 31 + rest)
    share = [math.exp(r.gauss(0.0, 1.0)) for _ in range(n)]
    each = [1 + int((rest - n) * s / sum(share)) for s in share]
    return [case["largest"]] + [min(x, case["largest"]) for x in each]


def _decays(case):
    """Weight decay per tensor: norm weights and biases (the small ones) have none."""
    return [0.1 if x > 4096 else 0.0 for x in _sizes(case)]


def work(case):
    op = case["op"]
    if op == "attn":
        e = _BYTES[case["dtype"]]
        lq, lk = _lengths(case)
        seen = sum(min(n, m + case["window"] - 1) + min(case["sinks"], max(0, n - m - case["window"] + 1))
                   for m, n in zip(lq, lk))   # keys that any query sees
        q = sum(lq) * case["heads"] * case["dim"] * e
        kv = 2 * seen * case["kv"] * case["dim"] * e
        lse = sum(lq) * case["heads"] * 4
        f = 2.0 * _pairs(case) * case["heads"] * case["dim"]
        if case["train"]:   # also the output's gradient in, the gradients out
            return {"bytes": 4 * q + 2 * kv + lse, "flops": 7 * f}
        return {"bytes": 2 * q + kv + lse, "flops": 2 * f}
    if op == "adamw":
        n, copy = sum(_sizes(case)), _BYTES.get(case["copy"], 0)
        state = 16 if case["bits"] == 32 else 4 + 16 / _BLOCK
        return {"bytes": n * (8 + _BYTES[case["grad"]] + copy + state), "flops": 15.0 * n}
    rows = case["batch"] * case["tokens"] * (case["heads"] + case["kv"])
    n, e = rows * case["dim"], _BYTES[case["dtype"]]
    if op == "rotary":
        return {"bytes": n * e * (4 if case["train"] else 2), "flops": n * (6.0 if case["train"] else 3.0)}
    stat = 4 * rows
    return {"bytes": n * e * (5 if case["train"] else 2) + stat, "flops": n * (18.0 if case["train"] else 7.0)}


# ----------------------------------------------------------------- inputs ----

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _frequencies(case):
    """(rot / 2 frequencies in 64 bits, s)."""
    rot, factor = case["rot"], case["factor"]
    base = 10000.0
    if case["scaling"] == "base":
        base *= factor ** (rot / (rot - 2))
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "ramp":
        keep = np.clip((f * 32768 / (2 * math.pi) - 1) / (32 - 1), 0.0, 1.0)
        return f * keep + f / factor * (1 - keep), 1.0 + 0.1 * math.log(factor)
    return f, 1.0


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(case)
    op = case["op"]
    if op == "adamw":
        return _prepare_adamw(s, case, seed, randn)
    dt = _DT[case["dtype"]]
    if op == "attn":
        h, kv, d, b = case["heads"], case["kv"], case["dim"], case["batch"]
        nq, nk = _lengths(case)
        s["scale"] = d ** -0.5
        s["max_q"], s["max_k"] = max(nq), max(nk)
        packed = case["lengths"] == "packed"
        lead_q, lead_k = ((case["q"],), (case["k"],)) if packed else ((b, case["q"]), (b, case["k"]))
        ints = dict(dtype=torch.int32, device=dev)
        s["start"] = torch.tensor(np.concatenate([[0], np.cumsum(nq)]), **ints) if packed else None
        s["q_lens"] = torch.tensor(nq, **ints) if case["lengths"] == "padded" else None
        s["k_lens"] = torch.tensor(nk, **ints) if case["lengths"] == "padded" else None
        if lead_q == lead_k:   # one projection's output: q, k and v are strided views of it
            s["q"], s["k"], s["v"] = randn(*lead_q, h + 2 * kv, d).to(dt).split([h, kv, kv], dim=-2)
        else:
            s["q"] = randn(*lead_q, h, d).to(dt)
            s["k"], s["v"] = randn(*lead_k, 2 * kv, d).to(dt).split([kv, kv], dim=-2)
        if case["train"]:
            s["dout"] = randn(*lead_q, h, d).to(dt)
        return s
    b, t, h, kv, d = case["batch"], case["tokens"], case["heads"], case["kv"], case["dim"]
    s["q"], s["k"], _ = (1.5 * randn(b, t, h + 2 * kv, d)).to(dt).split([h, kv, kv], dim=-2)
    s["positions"], s["first"] = None, case["far"]
    if case["at"] == "list":   # new tokens of many sequences, or documents that start anywhere
        start = torch.randint(0, case["far"], (b, 1 + t // 64), generator=g, device=dev)
        s["positions"] = (start.repeat_interleave(64, 1)[:, :t] + torch.arange(t, device=dev) % 64).int()
        s["first"] = 0
    s["freq"], s["amp"] = _frequencies(case)
    s["freq_dev"] = torch.from_numpy(s["freq"]).to(dev)
    if case["train"]:
        s["dq"], s["dk"] = randn(b, t, h, d).to(dt), randn(b, t, kv, d).to(dt)
    if op == "norm":
        s["wq"], s["wk"] = 1 + 0.1 * randn(d), 1 + 0.1 * randn(d)
    if own:
        from matrix_optimizer_step_02_amd import train
        s["rope"] = train.Rotary(s["freq"], layout=case["layout"], scale=s["amp"], device=dev)
    return s


def _prepare_adamw(s, case, seed, randn):
    sizes, total, dev = _sizes(case), sum(_sizes(case)), _device()

    def cut(flat):   # tensors one after the other in one buffer, as a program with flat buffers holds them
        return list(flat.split(sizes))

    s["W"] = cut(0.02 * randn(total))
    s["G"] = cut((1e-2 * randn(total)).to(_DT[case["grad"]]))
    s["decay"], s["t"], s["seed"] = _decays(case), 100, seed * 48271 + 1234567890123
    s["copy_to"] = None if case["copy"] == "none" else cut(torch.empty(total, dtype=_DT[case["copy"]], device=dev))
    s["max_norm"] = 0.5 * 1e-2 * total ** 0.5 if case["clip"] else 0.0
    s["m_scale"] = s["v_scale"] = None
    if case["bits"] == 32:
        s["m"], s["v"] = cut(1e-3 * randn(total)), cut((1e-3 * randn(total)).square_())
    else:
        blocks = [-(-x // _BLOCK) for x in sizes]
        # codes as a long run leaves them: m around zero, v positive; a scale per block
        s["m"] = cut((40 * randn(total)).clamp_(-240, 240).to(torch.float8_e4m3fn))
        s["v"] = cut((1000 * randn(total)).square_().clamp_(2.0 ** -10, 30000).to(torch.float8_e5m2))
        s["m_scale"] = list(torch.full((sum(blocks),), 2.0 ** -14, device=dev).split(blocks))
        s["v_scale"] = list(torch.full((sum(blocks),), 2.0 ** -36, device=dev).split(blocks))
    if own:
        import matrix_optimizer_step_02_amd as mo
        keys = ["W", "G", "m", "v"] + (["m_scale", "v_scale"] if case["bits"] == 8 else [])
        params = [{k: s[k][i] for k in keys} | {"weight_decay": s["decay"][i]} for i in range(len(sizes))]
        if s["copy_to"]:
            params = [p | {"W16": c} for p, c in zip(params, s["copy_to"])]
        s["group"] = mo.AdamWGroup(params, mo.AdamWHyper(**_ADAM))
        s["group"].t = s["t"]
    return s


# ------------------------------------------------------------ plain forms ----

def _angles(s):
    """cos and sin of every token and pair, 32 bits, from angles in 64: (batch, tokens, 1, rot / 2)."""
    if s["positions"] is None:
        p = (s["first"] + torch.arange(s["tokens"], device=s["q"].device)).expand(s["batch"], -1)
    else:
        p = s["positions"]
    a = (p.double()[..., None] * s["freq_dev"])[:, :, None]
    return (a.cos() * s["amp"]).float(), (a.sin() * s["amp"]).float()


def _turn(x, cos, sin, s):
    rot, half = s["rot"], s["rot"] // 2
    if s["layout"] == "half":
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rotary(s):
    dt = s["q"].dtype
    cos, sin = _angles(s)
    out = {n: _turn(s[n].float(), cos, sin, s).to(dt) for n in "qk"}
    if s["train"]:
        out |= {n: _turn(s[n].float(), cos, -sin, s).to(dt) for n in ("dq", "dk")}
    return out


def _plain_norm(s):
    dt = s["q"].dtype
    cos, sin = _angles(s)
    out = {}
    for n, w, d in (("q", s["wq"], "dq"), ("k", s["wk"], "dk")):
        x = s[n].float()
        rstd = (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        xh = x * rstd
        out[n], out[n + "_rstd"] = _turn(xh * w, cos, sin, s).to(dt), rstd[..., 0]
        if s["train"]:
            g = _turn(s[d].float(), cos, -sin, s)
            z = g * w
            out[d] = ((z - xh * (z * xh).mean(-1, keepdim=True)) * rstd).to(dt)
            out["dw" + n] = (g * xh).sum((0, 1, 2))
    return out


def _pad(x, start, most):
    """Packed rows (N, heads, dim) as (batch, most, heads, dim) and each slot's row (N where there is none)."""
    n = x.shape[0]
    row = start[:-1, None].long() + torch.arange(most, device=x.device)
    row = torch.where(row < start[1:, None].long(), row, n)
    return x[row.clamp(max=n - 1)], row


def _unpad(x, row, n):
    """(batch, most, ...) back to n packed rows; slots without a row go to one that is cut off."""
    out = torch.empty(n + 1, *x.shape[2:], dtype=x.dtype, device=x.device)
    out[row.reshape(-1)] = x.reshape(-1, *x.shape[2:])
    return out[:n]


def _plain_attention(s):
    q, k, v = (s[n].float() for n in "qkv")
    dev, dt, packed = q.device, s["q"].dtype, s["lengths"] == "packed"
    n, row = q.shape[0], None
    if packed:
        (q, row), (k, _), (v, _) = (_pad(x, s["start"], s["max_q"]) for x in (q, k, v))
        lq = lk = (s["start"][1:] - s["start"][:-1]).long().view(-1, 1, 1)
    elif s["lengths"] == "padded":
        lq, lk = s["q_lens"].long().view(-1, 1, 1), s["k_lens"].long().view(-1, 1, 1)
    else:
        lq, lk = (torch.full((1, 1, 1), x.shape[1], device=dev) for x in (q, k))
    group = s["heads"] // s["kv"]
    q = q.transpose(1, 2).contiguous()
    k, v = (x.transpose(1, 2).repeat_interleave(group, dim=1) for x in (k, v))
    i = torch.arange(q.shape[2], device=dev).view(1, -1, 1)
    j = torch.arange(k.shape[2], device=dev).view(1, 1, -1)
    last = i + lk - lq
    see = ((i < lq) & (j < lk) & (j <= last) & ((j > last - s["window"]) | (j < s["sinks"]))).unsqueeze(1)
    p = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(s["scale"]).masked_fill_(~see, -math.inf)
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    p = p.div_(torch.where(total > 0, total, 1.0))
    out = torch.matmul(p, v)

    def back(x):
        x = x.transpose(1, 2)
        return (_unpad(x, row, n) if packed else x).to(dt)

    lse = _unpad(lse.transpose(1, 2), row, n).t().contiguous() if packed else lse.transpose(0, 1).reshape(s["heads"], -1)
    if not s["train"]:
        return {"out": back(out), "lse": lse}
    do = s["dout"].float()
    do = (_pad(do, s["start"], s["max_q"])[0] if packed else do).transpose(1, 2).contiguous()
    dv = torch.matmul(p.transpose(-1, -2), do)
    dp = torch.matmul(do, v.transpose(-1, -2).contiguous())
    ds = dp.sub_((dp * p).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(-1, -2), q)
    dk, dv = (x.reshape(x.shape[0], s["kv"], group, *x.shape[2:]).sum(2) for x in (dk, dv))
    return {"out": back(out), "lse": lse, "dq": back(dq), "dk": back(dk), "dv": back(dv)}


def _random16(index, tensor, seed, offset):
    """16 bits for each eight elements of group ``index`` of tensor ``tensor``: (groups, 8)."""
    low = 0xFFFFFFFF
    c0, c1 = index, tensor
    c2, c3 = torch.full_like(c0, offset & low), torch.full_like(c0, offset >> 32 & low)
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & low) ^ c1 ^ k0, b & low, (a >> 32 & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((c0, c1, c2, c3), -1).int()
    return torch.stack((words & 0xFFFF, words >> 16 & 0xFFFF), -1).flatten(-2)


def _encode(y, r, digits, bias):
    """Magnitudes in 32 bits to 8-bit codes with ``digits`` mantissa bits, rounded by the 16 random bits r."""
    normal = (y.view(torch.int32) + (r << (7 - digits)) >> (23 - digits)) - ((127 - bias) << digits)
    small = (y * 2.0 ** (bias - 1 + digits + 16)).clamp(max=2.0 ** 24).int() + r >> 16
    return torch.where(y < 2.0 ** (1 - bias), small, normal)


def _blockwise(x, r, digits, bias, top, kind):
    """(codes of the type ``kind``, scales) of (blocks, 256) values; the largest magnitude is put below 2^(top + 1)."""
    e = (x.abs().amax(1).view(torch.int32) >> 23) - 127 - top
    e = e.clamp(-120, 120)
    scale = ((e + 127) << 23).view(torch.float32)
    code = _encode(x.abs() * ((127 - e) << 23).view(torch.float32)[:, None], r, digits, bias)
    return (code + (x < 0) * 128).to(torch.uint8).view(kind), scale


def _moments(m, v, g):
    m = m * _ADAM["beta1"] + g * (1 - _ADAM["beta1"])
    v = v * _ADAM["beta2"] + g * g * (1 - _ADAM["beta2"])
    return m, v


def _weights(W, m, v, t, decay):
    c1, c2 = 1 / (1 - _ADAM["beta1"] ** t), (1 - _ADAM["beta2"] ** t) ** -0.5
    den = torch._foreach_add(torch._foreach_mul(torch._foreach_sqrt(v), c2), _ADAM["eps"])
    step = torch._foreach_add(torch._foreach_div(torch._foreach_mul(m, c1), den), torch._foreach_mul(W, decay))
    torch._foreach_add_(W, torch._foreach_mul(step, -_ADAM["lr"]))


def _blocks(xs, dt=torch.float32):
    """Tensors as rows of 256, the last row of each filled up with zeros."""
    return torch.cat([torch.nn.functional.pad(x.to(dt), (0, -x.numel() % _BLOCK)) for x in xs]).view(-1, _BLOCK)


def _unblocks(rows, xs):
    """Rows of 256 back to tensors of the sizes of xs."""
    parts = rows.view(-1).split([x.numel() + -x.numel() % _BLOCK for x in xs])
    return [p[:x.numel()] for p, x in zip(parts, xs)]


def _plain_adamw(s):
    s["t"] += 1
    out = {}
    G = [g.float() for g in s["G"]]
    if s["clip"]:
        norm = torch.stack([g.double().square().sum() for g in G]).sum().sqrt()
        factor = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
        out["norm"] = norm.float()
        G = torch._foreach_mul(G, factor)
    if s["bits"] == 32:
        b1, b2 = _ADAM["beta1"], _ADAM["beta2"]
        m = torch._foreach_add(torch._foreach_mul(s["m"], b1), torch._foreach_mul(G, 1 - b1))
        v = torch._foreach_add(torch._foreach_mul(s["v"], b2), torch._foreach_mul(torch._foreach_mul(G, G), 1 - b2))
        _weights(s["W"], m, v, s["t"], s["decay"])
        torch._foreach_copy_(s["m"], m)
        torch._foreach_copy_(s["v"], v)
    else:
        dev = G[0].device
        rows = [-(-x.numel() // _BLOCK) for x in G]
        index = torch.cat([torch.arange(32 * n, device=dev) for n in rows])
        tensor = torch.arange(len(rows), device=dev).repeat_interleave(
            torch.tensor(rows, device=dev) * 32, output_size=32 * sum(rows))
        r = _random16(index, tensor, s["seed"], s["t"]).view(-1, _BLOCK)
        m = _blocks(s["m"]) * torch.cat(s["m_scale"])[:, None]
        v = _blocks(s["v"]) * torch.cat(s["v_scale"])[:, None]
        m, v = _moments(m, v, _blocks(G))
        _weights(s["W"], _unblocks(m, G), _unblocks(v, G), s["t"], s["decay"])
        mc, ms = _blockwise(m, r >> 8 | (r & 255) << 8, 3, 7, 7, torch.float8_e4m3fn)
        vc, vs = _blockwise(v, r, 2, 15, 14, torch.float8_e5m2)
        bytes_ = lambda xs: [x.view(torch.uint8) for x in xs]  # noqa: E731
        torch._foreach_copy_(bytes_(s["m"]) + bytes_(s["v"]),
                             _unblocks(mc.view(torch.uint8), G) + _unblocks(vc.view(torch.uint8), G))
        torch._foreach_copy_(s["m_scale"] + s["v_scale"], list(ms.split(rows)) + list(vs.split(rows)))
    if s["copy_to"]:
        torch._foreach_copy_(s["copy_to"], s["W"])
    return out | _state(s)


def _state(s):
    """The updated tensors, each kind as the buffer that all lie in."""
    keys = ["W", "m", "v"] + (["copy_to"] if s["copy_to"] else []) + (["m_scale", "v_scale"] if s["bits"] == 8 else [])
    return {k: s[k][0]._base for k in keys}


# ----------------------------------------------------------------- passes ----

def run(s):
    op = s["op"]
    if not own:
        return {"rotary": _plain_rotary, "norm": _plain_norm, "attn": _plain_attention, "adamw": _plain_adamw}[op](s)
    from matrix_optimizer_step_02_amd import train
    if op == "adamw":
        s["t"] += 1
        out, scale = {}, None
        if s["clip"]:
            clip = s["group"].grad_norm(s["max_norm"])
            out["norm"], scale = clip.norm, clip.scale
        s["group"].step(grad_scale=scale, rng=train.Rng(s["seed"], s["t"]) if s["bits"] == 8 else None)
        return out | _state(s)
    if op == "attn":
        how = dict(causal=True, window=s["window"], sinks=s["sinks"], scale=s["scale"])
        if s["lengths"] == "packed":
            how |= dict(q_start=s["start"], k_start=s["start"], max_q=s["max_q"], max_k=s["max_k"])
        elif s["lengths"] == "padded":
            how |= dict(q_lens=s["q_lens"], k_lens=s["k_lens"])
        out, lse = train.attention_forward(s["q"], s["k"], s["v"], **how)
        if not s["train"]:
            return {"out": out, "lse": lse}
        dq, dk, dv = train.attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, **how)
        return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    at = dict(positions=s["positions"], first=s["first"])
    if op == "rotary":
        q, k = train.rotary_forward(s["q"], s["k"], s["rope"], **at)
        out = {"q": q, "k": k}
        if s["train"]:
            out["dq"], out["dk"] = train.rotary_backward(s["dq"], s["dk"], s["rope"], **at)
        return out
    q, k, q_rstd, k_rstd = train.qk_norm_forward(s["q"], s["k"], s["wq"], s["wk"], eps=1e-6, rope=s["rope"], **at)
    out = {"q": q, "k": k, "q_rstd": q_rstd, "k_rstd": k_rstd}
    if s["train"]:
        out["dq"], out["dk"], out["dwq"], out["dwk"] = train.qk_norm_backward(
            s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], q_rstd, k_rstd, rope=s["rope"], **at)
    return out


# ---------------------------------------------------------------- 64 bits ----

def _exact_attention(case, s):
    q, k, v = (s[n].double() for n in "qkv")
    dev = q.device
    nq, nk = _lengths(case)
    h, kv, d = case["heads"], case["kv"], case["dim"]
    group = h // kv
    flat_q, flat_k, flat_v = q.reshape(-1, h, d), k.reshape(-1, kv, d), v.reshape(-1, kv, d)
    out, dq = torch.zeros_like(flat_q), torch.zeros_like(flat_q)
    dk, dv = torch.zeros_like(flat_k), torch.zeros_like(flat_v)
    lse = torch.full((h, flat_q.shape[0]), -math.inf, dtype=torch.float64, device=dev)
    do = s["dout"].double().reshape(flat_q.shape) if case["train"] else None
    a = c = 0
    for n, (m, w) in enumerate(zip(nq, nk)):
        if case["lengths"] != "packed":
            a, c = n * case["q"], n * case["k"]
        key, last = torch.arange(w, device=dev)[None], torch.arange(m, device=dev)[:, None] + (w - m)
        hide = (key > last) | ((key <= last - case["window"]) & (key >= case["sinks"]))
        for x in range(h):
            qs, ks, vs = flat_q[a:a + m, x], flat_k[c:c + w, x // group], flat_v[c:c + w, x // group]
            sc = torch.where(hide, -math.inf, qs @ ks.t().contiguous() * s["scale"])
            z = torch.logsumexp(sc, 1)
            lse[x, a:a + m] = z
            p = torch.where(hide, 0.0, (sc - torch.where(z.isinf(), 0.0, z)[:, None]).exp())
            o = p @ vs
            out[a:a + m, x] = o
            if do is not None:
                g = do[a:a + m, x]
                dp = g @ vs.t().contiguous()   # a row of one key: dp - dp p is zero to the bit
                ds = p * (dp - (dp * p).sum(1, keepdim=True)) * s["scale"]
                dq[a:a + m, x] = ds @ ks
                dk[c:c + w, x // group] += ds.t().contiguous() @ qs
                dv[c:c + w, x // group] += p.t().contiguous() @ g
        a, c = a + m, c + w
    got = {"out": out.view(q.shape), "lse": lse}
    if do is not None:
        got |= {"dq": dq.view(q.shape), "dk": dk.view(k.shape), "dv": dv.view(v.shape)}
    return got


def _exact_turn(x, s, back):
    """The rotation as a product of complex numbers, in 64 bits."""
    b, t, rot = x.shape[0], x.shape[1], s["rot"]
    p = s["positions"]
    p = torch.arange(s["first"], s["first"] + t, device=x.device).expand(b, t) if p is None else p
    angle = p.to(torch.float64).unsqueeze(-1) * torch.from_numpy(s["freq"]).to(x.device)
    e = torch.polar(torch.full_like(angle, s["amp"]), -angle if back else angle).unsqueeze(2)
    y = x.clone()
    if s["layout"] == "half":
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * e
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.view_as_complex(x[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * e
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    return y


def _exact_norm(s):
    got = {}
    for n, w, d in (("q", s["wq"].double(), "dq"), ("k", s["wk"].double(), "dk")):
        x = s[n].double()
        rms = torch.sqrt(x.pow(2).mean(-1) + 1e-6)
        xh = x / rms[..., None]
        got[n], got[n + "_rstd"] = _exact_turn(xh * w, s, False), 1 / rms
        if s["train"]:
            g = _exact_turn(s[d].double(), s, True)
            along = (g * w * xh).mean(-1, keepdim=True)
            got[d] = (g * w - along * xh) / rms[..., None]
            got["dw" + n] = torch.einsum("bthd,bthd->d", g, xh)
    return got


def _exact_bits(n, tensor, seed, offset):
    """16 random bits of each of a tensor's n elements, by unsigned 64-bit products on the host."""
    u = np.uint64
    low, half = u(0xFFFFFFFF), u(32)
    groups = -(-n // 8)
    got = np.empty((groups, 4), dtype="<u4")
    for a in range(0, groups, 1 << 21):
        e = min(groups, a + (1 << 21))
        x = [np.arange(a, e, dtype=u)] + [np.full(e - a, c, dtype=u) for c in (tensor, offset & 0xFFFFFFFF, offset >> 32)]
        for i in range(10):
            key = [u((seed + i * 0x9E3779B9) & 0xFFFFFFFF), u(((seed >> 32) + i * 0xBB67AE85) & 0xFFFFFFFF)]
            p0, p1 = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
            x = [(p1 >> half) ^ x[1] ^ key[0], p1 & low, (p0 >> half) ^ x[3] ^ key[1], p0 & low]
        for w in range(4):
            got[a:e, w] = x[w]
    return got.view("<u2").reshape(-1)[:n].astype(np.int32)


def _exact_codes(x, bits, digits, bias, top):
    """(values that the codes stand for, without the scale; scales): the grid around each value, in 64 bits."""
    pad = -x.numel() % _BLOCK
    b = torch.nn.functional.pad(x, (0, pad)).view(-1, _BLOCK)
    most = b.abs().amax(1)
    power = torch.where(most > 0, torch.floor(torch.log2(most.clamp(min=1e-300))) - top, -120.0).clamp(-120, 120)
    y = (b.abs() * torch.exp2(-power)[:, None]).view(-1)[:x.numel()]
    grid = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** (1 - bias)))) - digits)
    return torch.sign(x) * torch.floor(y / grid + bits / 65536) * grid, torch.exp2(power)


def _exact_adamw(case, s):
    t, b1, b2 = s["t"] + 1, _ADAM["beta1"], _ADAM["beta2"]
    got = {k: [] for k in _state(s)}
    factor = 1.0
    if case["clip"]:
        norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in s["G"]))
        factor = min(1.0, s["max_norm"] / (norm + 1e-6))
    for i, g in enumerate(s["G"]):
        g, w, m, v = g.double() * factor, s["W"][i].double(), s["m"][i].double(), s["v"][i].double()
        if case["bits"] == 8:
            m = m * s["m_scale"][i].double().repeat_interleave(_BLOCK)[:m.numel()]
            v = v * s["v_scale"][i].double().repeat_interleave(_BLOCK)[:v.numel()]
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g ** 2
        update = m / (1 - b1 ** t) / (torch.sqrt(v / (1 - b2 ** t)) + _ADAM["eps"])
        w = w - _ADAM["lr"] * (update + s["decay"][i] * w)
        if case["bits"] == 8:
            r = torch.from_numpy(_exact_bits(m.numel(), i, s["seed"], t)).to(w.device)
            m, scale = _exact_codes(m, (r & 255) * 256 + r // 256, 3, 7, 7)
            got["m_scale"].append(scale)
            v, scale = _exact_codes(v, r, 2, 15, 14)
            got["v_scale"].append(scale)
        for k, x in (("W", w), ("m", m), ("v", v), ("copy_to", w)):
            if k in got:
                got[k].append(x)
    got = {k: torch.cat(x) for k, x in got.items()}
    return got | ({"norm": norm} if case["clip"] else {})


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attn":
        return _exact_attention(case, s)
    if op == "adamw":
        return _exact_adamw(case, s)
    if op == "norm":
        return _exact_norm(s)
    got = {n: _exact_turn(s[n].double(), s, False) for n in "qk"}
    if case["train"]:
        got |= {n: _exact_turn(s[n].double(), s, True) for n in ("dq", "dk")}
    return got
