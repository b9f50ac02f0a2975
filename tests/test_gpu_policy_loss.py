"""GPU tests of the clipped policy loss against the fp64 oracle.

The exponentials' arguments carry a relative error of 3 2^-24 of at most 100
(in base 2), and a sum of V exponentials at most 192 2^-24 of itself (a thread
adds at most 160 in turn, a tree the rest): lse and logp are within 2e-5,
probabilities and exp(logp - old) within 5e-5 of themselves, and a gradient
k (onehot - p) within 2e-4 of |k| (onehot + p) plus the output's rounding u.
"""

import numpy as np
import pytest

from oracle import train_ops as T

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _train():
    from matrix_optimizer_step_02_amd import train
    return train


U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def np64(t):
    return t.detach().double().cpu().numpy()


def make(rows, vocab, dtype, seed=0, i64=False, scale=1.0):
    torch = _torch()
    dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (2 * torch.randn(rows, vocab, generator=g, device="cuda")).to(dt)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int64 if i64 else torch.int32)
    x[torch.arange(rows), t.long()] += 5
    z = x.double() * scale
    logp = (z.gather(1, t.long()[:, None])[:, 0] - z.logsumexp(1)).float()
    gap = torch.tensor([0.0, 0.1, -0.1, 0.5, -0.5, 2.0, -2.0], device="cuda").repeat(rows // 7 + 1)[:rows]
    old, ref = logp - gap, logp + 0.3 * torch.randn(rows, generator=g, device="cuda")
    adv = torch.randn(rows, generator=g, device="cuda")
    w = torch.rand(rows, generator=g, device="cuda") / rows
    if rows > 3:
        w[1::5] = 0
    return x, t, old, ref, adv, w


def compare(got, x, t, old, ref, adv, w, dtype, kl, scale, grad=1.0, lo=0.2, hi=0.28):
    r = T.policy_loss(np64(x), t.cpu().numpy(), np64(old), np64(ref), np64(adv), np64(w), lo, hi, kl, scale, grad)
    terms = np.abs(r["term"])
    # a term's own error: r within 5e-5, and the KL term's derivative |1 - e^d| times logp's 2e-5
    slack = (2e-4 * (terms + np.abs(r["slope"])) + np.abs(np64(w)) * kl * 1e-5).sum() + 1e-12
    assert abs(float(got["loss"]) - r["loss"]) <= slack
    assert np.max(np.abs(np64(got["logp"]) - r["logp"])) <= 2e-5
    if "lse" in got:
        assert np.max(np.abs(np64(got["lse"]) - r["lse"])) <= 2e-5
        assert np.max(np.abs(np64(got["slope"]) - r["slope"]) - 2e-4 * (np.abs(r["slope"]) + kl * np.abs(np64(w)))) <= 0
    d, ref_d = np64(got["dlogits"]), r["dlogits"]
    n = np.arange(len(t))
    hot = np.zeros_like(d)
    hot[n, np.clip(t.cpu().numpy(), 0, d.shape[1] - 1)] = 1
    k = np.abs(grad * scale) * (np.abs(r["slope"]) + kl * np.abs(np64(w)))[:, None]
    p = np.exp(scale * np64(x) - r["lse"][:, None])
    tiny = 2.0 ** -25 if dtype == "f16" else 0
    assert np.max(np.abs(d - ref_d) - (U[dtype] * np.abs(ref_d) + 2e-4 * k * (hot + p) + tiny + 1e-30)) <= 0


SIZES = [(1, 1), (5, 2), (9, 7), (30, 8), (33, 1000), (20, 4096), (11, 4097), (9, 8193), (8, 16385), (6, 32769), (3, 65537),
         (2, 81921), (3, 131072), (2, 131073), (2, 163841)]


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_step_and_forward_backward(rows, vocab, dtype):
    torch, train = _torch(), _train()
    print(f"policy {rows}x{vocab} {dtype}", flush=True)
    kl, scale = (0.1, 0.7) if rows % 2 else (0.0, 1.0)
    x, t, old, ref, adv, w = make(rows, vocab, dtype, seed=vocab, i64=rows % 3 == 0, scale=scale)
    how = dict(clip_low=0.2, clip_high=0.28, kl_coef=kl, logit_scale=scale, ref_logp=ref if kl else None)
    loss, logp, d = train.policy_loss_step(x, t, old, adv, w, grad=2.0, **how)
    compare({"loss": loss, "logp": logp, "dlogits": d}, x, t, old, ref, adv, w, dtype, kl, scale, grad=2.0)
    f = train.policy_loss_forward(x, t, old, adv, w, **how)
    d = train.policy_loss_backward(x, t, f, grad=torch.tensor(0.5, device="cuda"), logit_scale=scale)
    compare({"loss": f.loss, "logp": f.logp, "lse": f.lse, "slope": f.slope, "dlogits": d}, x, t, old, ref, adv, w, dtype,
            kl, scale, grad=0.5)
    assert torch.equal(f.loss, loss) and torch.equal(f.logp, logp)


@pytest.mark.parametrize("vocab", [100, 5000, 170001])
def test_in_place_and_strided(vocab):
    torch, train = _torch(), _train()
    print(f"policy in place {vocab}", flush=True)
    x, t, old, ref, adv, w = make(6, vocab, "bf16")
    how = dict(ref_logp=ref, kl_coef=0.1)
    loss, logp, d = train.policy_loss_step(x, t, old, adv, w, **how)
    wide = torch.full((6, vocab + 13), float("nan"), device="cuda", dtype=torch.bfloat16)
    v = wide[:, 3:3 + vocab]
    v.copy_(x)
    out = torch.full((6, vocab + 5), 7.0, device="cuda", dtype=torch.bfloat16)
    loss2, logp2, d2 = train.policy_loss_step(v, t, old, adv, w, out=out[:, 2:2 + vocab], **how)
    assert torch.equal(loss, loss2) and torch.equal(logp, logp2) and torch.equal(d, d2)
    assert (out[:, :2] == 7).all() and (out[:, 2 + vocab:] == 7).all()
    f = train.policy_loss_forward(x, t, old, adv, w, **how)
    y = x.clone()
    train.policy_loss_backward(y, t, f, out=y)
    z = x.clone()
    assert train.policy_loss_step(z, t, old, adv, w, out=z, **how)[2] is z
    assert torch.equal(z, d)
    assert (y.float() - d.float()).abs().max() <= 2.0 ** -7 * d.float().abs().max()


@pytest.mark.parametrize("vocab", [1000, 40000, 170001])
def test_rows_left_out_may_hold_anything(vocab):
    torch, train = _torch(), _train()
    print(f"policy masked {vocab}", flush=True)
    x, t, old, ref, adv, w = make(10, vocab, "f32", i64=True)
    want = train.policy_loss_step(x, t, old, adv, w, ref_logp=ref, kl_coef=0.1)
    out = w == 0
    x[out], t[out], old[out], ref[out], adv[out] = float("nan"), -100, float("nan"), float("inf"), float("nan")
    got = train.policy_loss_step(x, t, old, adv, w, ref_logp=ref, kl_coef=0.1)
    f = train.policy_loss_forward(x, t, old, adv, w, ref_logp=ref, kl_coef=0.1)
    d = train.policy_loss_backward(x, t, f)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and (got[2][out] == 0).all()
    assert torch.equal(f.loss, want[0]) and (d[out] == 0).all() and not d.isnan().any()


@pytest.mark.parametrize("vocab", [1000, 170001])
def test_infinite_logits_and_bad_targets(vocab):
    """-inf hides a token (gradient 0); NaN, and a target outside the vocabulary, make their rows and the loss NaN."""
    torch, train = _torch(), _train()
    print(f"policy infinities {vocab}", flush=True)
    x, t, old, ref, adv, w = make(4, vocab, "f32")
    w[:] = 0.25
    x[:, 5:300] = -float("inf")
    x[torch.arange(4), t.long()] = 3.0
    loss, logp, d = train.policy_loss_step(x, t, old, adv, w)
    compare({"loss": loss, "logp": logp, "dlogits": d}, x, t, old, ref, adv, w, "f32", 0.0, 1.0, hi=0.2)
    for bad in ("target", "negative", "nan", "all -inf"):
        y, s = x.clone(), t.clone()
        if bad == "target":
            s[2] = vocab
        elif bad == "negative":
            s[2] = -1
        elif bad == "nan":
            y[2, 7] = float("nan")
        else:
            y[2] = -float("inf")
        f = train.policy_loss_forward(y, s, old, adv, w)
        g = train.policy_loss_backward(y, s, f)
        loss, logp, d = train.policy_loss_step(y, s, old, adv, w)
        for row in range(4):
            assert bool(logp[row].isnan()) == (row == 2) and bool(f.logp[row].isnan()) == (row == 2), bad
            assert bool(d[row].isnan().all()) == (row == 2) and bool(g[row].isnan().all()) == (row == 2), bad
            assert bool(d[row].isnan().any()) == (row == 2), bad
        assert loss.isnan() and f.loss.isnan()


def test_no_rows_and_equal_bits():
    torch, train = _torch(), _train()
    print("policy empty, streams, graph", flush=True)
    v = torch.zeros(0, device="cuda")
    loss, logp, d = train.policy_loss_step(torch.zeros(0, 9, device="cuda"), torch.zeros(0, device="cuda", dtype=torch.int32), v, v, v)
    assert float(loss) == 0 and d.shape == (0, 9)
    x, t, old, ref, adv, w = make(300, 3001, "bf16")
    how = dict(ref_logp=ref, kl_coef=0.1)
    first = train.policy_loss_step(x, t, old, adv, w, **how)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = train.policy_loss_step(x, t, old, adv, w, stream=s, **how)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = train.policy_loss_step(x, t, old, adv, w, **how)
    for n in range(3):
        x.copy_(torch.randn_like(x))
        g.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in held]
        assert all(torch.equal(a, b) for a, b in zip(got, train.policy_loss_step(x, t, old, adv, w, **how))), n


def test_more_rows_than_one_launch_holds():
    """Past 2^31 threads the rows take several launches: the last rows are as
    they are alone, and so are the first."""
    torch, train = _torch(), _train()
    rows, vocab = 2 ** 23 + 5, 9
    print("policy rows", rows, flush=True)
    x, t, old, _, adv, w = (a[:4096] if a is not None else None for a in make(4096, vocab, "bf16"))
    often = lambda a: a.repeat(rows // 4096 + 1, *[1] * (a.dim() - 1))[:rows]  # noqa: E731
    many = [often(a) for a in (x, t, old, adv, w)]
    few = train.policy_loss_step(x, t, old, adv, w)
    loss, logp, d = train.policy_loss_step(*many)
    f = train.policy_loss_forward(*many)
    g = train.policy_loss_backward(many[0], many[1], f)
    for a in (logp, f.logp):
        assert torch.equal(a, often(few[1]))
    assert torch.equal(d, often(few[2]))
    # the two calls' probabilities are the same to the bit, their gradients to two roundings
    assert torch.equal(g[-5:], g[:5]) and torch.equal(g, often(g[:4096]))
    want = float(few[0]) * (rows // 4096) + float(train.policy_loss_step(x[:5], t[:5], old[:5], adv[:5], w[:5])[0])
    assert abs(float(loss) - want) <= 2 ** -22 * abs(want) + 1e-30 and torch.equal(loss, f.loss)


@pytest.mark.parametrize("rows", [16384, 16385, 40001])
def test_sum_of_many_rows(rows):
    """The terms' sum is 64-bit wherever it is split: off by one rounding to 32."""
    torch, train = _torch(), _train()
    print("policy sum", rows, flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, 17, generator=g, device="cuda")
    t = torch.zeros(rows, device="cuda", dtype=torch.int32)
    adv = torch.randn(rows, generator=g, device="cuda")
    one = torch.ones(rows, device="cuda")
    old = train.policy_loss_forward(x, t, one, adv, one).logp   # ratio exp(0) = 1: the terms are -adv to the bit
    loss = float(train.policy_loss_forward(x, t, old, adv, one).loss)
    want = float(-adv.double().sum())
    assert abs(loss - want) <= 2.0 ** -24 * abs(want) + rows * 2.0 ** -53 * float(adv.double().abs().sum())


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 9])
@pytest.mark.parametrize("vocab", [1, 8, 505, 1024, 1025, 2047, 2048, 2049])
def test_small_vocabularies(rows, vocab):
    """Rows of a wavefront share workgroups: the last ones are not full."""
    torch, train = _torch(), _train()
    print("policy small", rows, vocab, flush=True)
    x, t, old, ref, adv, w = make(rows, vocab, "bf16", seed=vocab + rows)
    loss, logp, d = train.policy_loss_step(x, t, old, adv, w, ref_logp=ref, kl_coef=0.1, clip_high=0.28)
    compare({"loss": loss, "logp": logp, "dlogits": d}, x, t, old, ref, adv, w, "bf16", 0.1, 1.0)
    f = train.policy_loss_forward(x, t, old, adv, w, ref_logp=ref, kl_coef=0.1, clip_high=0.28)
    d = train.policy_loss_backward(x, t, f)
    compare({"loss": f.loss, "logp": f.logp, "lse": f.lse, "slope": f.slope, "dlogits": d}, x, t, old, ref, adv, w, "bf16",
            0.1, 1.0)


@pytest.mark.parametrize("vocab", [1000, 5000, 170001])
@pytest.mark.parametrize("bad", ["old", "advantage", "reference", "weight"])
def test_nan_of_a_rows_inputs_reaches_its_results(vocab, bad):
    """One NaN makes its row's slope and gradient and the loss NaN, and leaves the other rows as they were."""
    torch, train = _torch(), _train()
    print(f"policy nan {bad} {vocab}", flush=True)
    x, t, old, ref, adv, w = make(4, vocab, "f32")
    w[:] = 0.25
    how = dict(ref_logp=ref, kl_coef=0.1)
    want = train.policy_loss_step(x, t, old, adv, w, **how)
    f0 = train.policy_loss_forward(x, t, old, adv, w, **how)
    g0 = train.policy_loss_backward(x, t, f0)
    {"old": old, "advantage": adv, "reference": ref, "weight": w}[bad][2] = float("nan")
    loss, logp, d = train.policy_loss_step(x, t, old, adv, w, **how)
    f = train.policy_loss_forward(x, t, old, adv, w, **how)
    g = train.policy_loss_backward(x, t, f)
    assert loss.isnan() and f.loss.isnan() and f.slope[2].isnan()
    assert d[2].isnan().all() and g[2].isnan().all()
    for n in (0, 1, 3):
        assert torch.equal(d[n], want[2][n]) and torch.equal(g[n], g0[n]) and f.slope[n] == f0.slope[n]
    assert torch.equal(logp, want[1])
    if bad == "reference":   # not read without a KL term
        assert torch.equal(train.policy_loss_step(x, t, old, adv, w, ref_logp=ref)[0],
                           train.policy_loss_step(x, t, old, adv, w)[0])


def test_no_advantage_is_no_term_whatever_the_ratio():
    """0 times a ratio past the range of fp32 is 0, as it is for every ratio."""
    torch, train = _torch(), _train()
    print("policy advantage 0", flush=True)
    x, t, old, ref, adv, w = make(3, 100, "f32")
    w[:], adv[1], old[1] = 0.5, 0.0, -200.0
    f = train.policy_loss_forward(x, t, old, adv, w)
    assert f.loss.isfinite() and f.slope[1] == 0
    assert not train.policy_loss_step(x, t, old, adv, w)[2][1].any()


@pytest.mark.parametrize("offset", [0.0, 100.0, 1000.0, -1000.0])
@pytest.mark.parametrize("vocab", [1000, 5000, 170001])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_a_common_offset_of_the_logits_costs_nothing(vocab, offset, dtype):
    """The softmax depends on differences of logits, so bounds do not grow with
    an offset. With u = 2^-24 and a sum of n terms in turn and in a tree: the
    sum is off by n u, an exponential by 4 u + 3 u |z - max| (the rounded
    difference, the rounded change of base and the instruction), the logarithm
    and what is done with it by 4 u of what it holds, which is below log V."""
    torch, train = _torch(), _train()
    print(f"policy offset {vocab} {offset} {dtype}", flush=True)
    scale, kl, lo, hi, u = float(np.float32(0.7)), 0.1, 0.2, 0.28, 2.0 ** -24
    added = {1000: 16 + 6, 5000: 32 + 10, 170001: 168 + 22}[vocab]
    g = torch.Generator(device="cuda").manual_seed(vocab)
    rows = 12
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    x = 2 * torch.randn(rows, vocab, generator=g, device="cuda")
    x[torch.arange(rows), t.long()] += torch.tensor([0.0, 12.0, 25.0, 45.0], device="cuda").repeat(3)
    x = (x + offset).to({"f32": torch.float32, "f16": torch.float16}[dtype])
    z = x.double() * scale
    true = z.gather(1, t.long()[:, None])[:, 0] - z.logsumexp(1)
    gap = torch.tensor([0.0, 0.1, -0.1, 0.5, -0.5, 2.0], device="cuda").repeat(2)
    old, ref = (true - gap).float(), (true + 0.3 * torch.randn(rows, generator=g, device="cuda")).float()
    adv, w = torch.randn(rows, generator=g, device="cuda"), torch.full((rows,), 1.0 / rows, device="cuda")
    how = dict(ref_logp=ref, kl_coef=kl, logit_scale=scale, clip_low=lo, clip_high=hi)
    loss, logp, d = train.policy_loss_step(x, t, old, adv, w, **how)
    f = train.policy_loss_forward(x, t, old, adv, w, **how)
    b = train.policy_loss_backward(x, t, f, logit_scale=scale)
    r = T.policy_loss(np64(x), t.cpu().numpy(), np64(old), np64(ref), np64(adv), np64(w), lo, hi, kl, scale)
    zc = np64(z)
    below = zc.max(1) - zc[np.arange(rows), t.cpu().numpy()]         # of the target, below the maximum
    p = np.exp(zc - r["lse"][:, None])
    mean = (p * (zc.max(1)[:, None] - zc)).sum(1)                    # what the terms' own errors weigh
    e_logp = u * (added + 4 + 3 * mean + 4 * np.log(vocab) + 4 * below + 4 * np.abs(r["logp"]))
    assert np.all(np.abs(np64(logp) - r["logp"]) <= e_logp) and (logp <= 0).all()
    assert torch.equal(f.logp, logp)
    assert np.all(np.abs(np64(f.lse) - r["lse"]) <= e_logp + u * np.abs(r["lse"]))
    # exp(logp - old) and exp(ref - logp): e_logp, the difference's rounding and the function's two steps
    ratio, back = np.exp(r["logp"] - np64(old)), np.exp(np64(ref) - r["logp"])
    wide = np64(w) * (np.abs(np64(adv)) * ratio + kl * back)
    e_slope = wide * (e_logp + 12 * u)
    assert np.all(np.abs(np64(f.slope) - r["slope"]) <= e_slope)
    assert abs(float(loss) - r["loss"]) <= (e_slope + np64(w) * kl * (e_logp + 4 * u)).sum() + u * abs(r["loss"]) + 8 * u * np.abs(r["term"]).sum()
    hot = np.zeros_like(p)
    hot[np.arange(rows), t.cpu().numpy()] = 1
    e_p = p * (e_logp[:, None] + u * (8 + 4 * np.abs(zc - r["lse"][:, None]))) + hot * 4 * u * (1 - p)
    tiny = 2.0 ** -25 if dtype == "f16" else 0
    for got in (d, b):
        err = np.abs(np64(got) - r["dlogits"])
        bound = scale * (e_slope[:, None] * np.abs(hot - p) + (np.abs(r["slope"]) + e_slope)[:, None] * e_p)
        bound += (U[dtype] + 4 * u) * (np.abs(r["dlogits"]) + bound) + tiny + 1e-37
        assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("vocab", [9, 1000, 5000, 40000, 170001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_the_types_lowest_value(vocab, dtype):
    """Logits masked by the type's lowest value: beside others they count for nothing, a row of nothing else is
    uniform; and finite logits far past the range of exact whole numbers keep their differences."""
    torch, train = _torch(), _train()
    print(f"policy lowest {vocab} {dtype}", flush=True)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    low = torch.finfo(dt).min
    x = torch.full((3, vocab), low, device="cuda", dtype=dt)
    x[1, 1:3] = 1.0
    x[2], x[2, 2] = 2.0 ** 40, 2.0 ** 40 + 2.0 ** 33
    t = torch.tensor([2, 2, 2], device="cuda", dtype=torch.int32)
    one, none = torch.ones(3, device="cuda"), torch.zeros(3, device="cuda")
    old = torch.tensor([-np.log(vocab), -np.log(2), 0.0], device="cuda", dtype=torch.float32)
    f = train.policy_loss_forward(x, t, old, one, one)
    g = train.policy_loss_backward(x, t, f)
    loss, logp, d = train.policy_loss_step(x, t, old, one, one)
    want = torch.zeros(3, vocab, device="cuda", dtype=torch.float64)   # slope -1: p - onehot
    want[0], want[1, 1:3] = 1 / vocab, 0.5
    want[0, 2] -= 1
    want[1, 2] -= 1
    # as in compare: logp within 2e-5, gradients within 2e-4 of themselves and the rounding
    assert ((logp.double().cpu() - old.double().cpu()).abs() <= 2e-5).all() and torch.equal(f.logp, logp)
    for got in (d, g):
        assert ((got.double() - want).abs() <= (2e-4 + U[dtype]) * want.abs() + 1e-12).all()
