"""GPU tests of attention (forward and backward) against the fp64 oracle.

Bounds, per element, with u = eps / 2 of the storage type. The kernels round
P (forward, and again for dV) and dS to that type, and the outputs; the scores
are fp32 sums of exact products, off by at most (d + 4) 2^-24 scale |q||k|,
which is below 2^-13 here and enters P relatively; 2^-12 covers it with the
exponential and the fp32 sums. float16 holds what is below 2^-14 in steps of
2^-24, so every rounding to it may be off by 2^-25: of probabilities, of score
gradients and of the outputs themselves.
  out: u |out| + (u + 2^-12) P |v| + 2^-25 sum |v| + 2^-25
  D:   dO . (error of the stored out), so |dO| . (2 u |out| + (u + 2^-12) P |v| ...)
  dS:  u |dS| + P dD + 2^-12 P (|dP| + |D|) + 2^-25
and those carried through the products with |k|, |q|, |dO|.
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


U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SLACK, TINY = 2.0 ** -12, 2.0 ** -25


def _dt(name):
    torch = _torch()
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def np64(t):
    return t.detach().double().cpu().numpy()


def worst(got, ref, bound):
    """Largest error over its bound; non-finite values must agree."""
    assert got.shape == ref.shape
    fin = np.isfinite(ref)
    assert np.array_equal(fin, np.isfinite(got)), "non-finite values differ"
    assert np.array_equal(got[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)])
    d = np.abs(got[fin] - ref[fin]) / (np.broadcast_to(bound, ref.shape)[fin] + TINY)
    return float(d.max()) if d.size else 0.0


def check_sequence(q, k, v, dout, got, scale, see, u):
    """One sequence: q, dout (nq, h, d); k, v (nk, hk, d); got a dict of fp64 arrays of the same layout."""
    heads, group = q.shape[1], q.shape[1] // k.shape[1]
    bounds = {n: np.zeros(x.shape) for n, x in (("dk", k), ("dv", v))}
    refs = {n: np.zeros(x.shape) for n, x in (("dk", k), ("dv", v))}
    for h in range(heads):
        kk, vv = k[:, h // group], v[:, h // group]
        r = T.attention(q[:, h], kk, vv, scale, see, None if dout is None else dout[:, h])
        e_out = u * np.abs(r["out"]) + (u + SLACK) * (r["p"] @ np.abs(vv)) + TINY * (see @ np.abs(vv))
        assert worst(got["out"][:, h], r["out"], e_out) <= 1
        e_lse = 2.0 ** -13 + 2.0 ** -21 * np.abs(np.where(np.isfinite(r["lse"]), r["lse"], 0))
        assert worst(got["lse"][h], r["lse"], e_lse) <= 1
        if dout is None:
            continue
        g = np.abs(dout[:, h])
        e_D = (g * (e_out + u * np.abs(r["out"]))).sum(1) + SLACK * np.abs(r["D"])
        e_ds = (u * np.abs(r["ds"]) + r["p"] * e_D[:, None] + SLACK * r["p"] * (np.abs(r["dp"]) + np.abs(r["D"])[:, None])
                + TINY * see)
        e_dq = u * np.abs(r["dq"]) + scale * e_ds @ np.abs(kk) + SLACK * scale * np.abs(r["ds"]) @ np.abs(kk)
        assert worst(got["dq"][:, h], r["dq"], e_dq) <= 1
        refs["dk"][:, h // group] += r["dk"]
        refs["dv"][:, h // group] += r["dv"]
        bounds["dk"][:, h // group] += scale * e_ds.T @ np.abs(q[:, h]) + SLACK * scale * np.abs(r["ds"]).T @ np.abs(q[:, h])
        bounds["dv"][:, h // group] += ((u + SLACK) * r["p"] + TINY * see).T @ g
    if dout is not None:
        for n in ("dk", "dv"):
            assert worst(got[n], refs[n], bounds[n] + u * np.abs(refs[n])) <= 1, n


def run(q, k, v, dout, **how):
    train, torch = _train(), _torch()
    out, lse = train.attention_forward(q, k, v, **how)
    got = {"out": out, "lse": lse}
    if dout is not None:
        got["dq"], got["dk"], got["dv"] = train.attention_backward(dout, q, k, v, out, lse, **how)
    torch.cuda.synchronize()
    return got


def dense(batch, nq, nk, heads, kv, d, dtype="bf16", causal=False, window=0, seed=0, scale=None, spread=1.0):
    torch = _torch()
    print(f"attention {batch}x{nq}x{nk} heads {heads}/{kv} d {d} {dtype} causal {causal} window {window}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(_dt(dtype))  # noqa: E731
    q, k, v, dout = spread * mk(batch, nq, heads, d), mk(batch, nk, kv, d), mk(batch, nk, kv, d), mk(batch, nq, heads, d)
    got = run(q, k, v, dout, causal=causal, window=window, scale=scale)
    got = {n: np64(t) for n, t in got.items()}
    see = T.visible(nq, nk, causal, window)
    lse = got["lse"].reshape(heads, batch, nq)
    for b in range(batch):
        one = {n: got[n][b] for n in ("out", "dq", "dk", "dv")} | {"lse": lse[:, b]}
        check_sequence(np64(q[b]), np64(k[b]), np64(v[b]), np64(dout[b]), one,
                       d ** -0.5 if scale is None else scale, see, U[dtype])


@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 64), (2, 3), (31, 33), (64, 64), (65, 127), (128, 128), (129, 200),
                                   (200, 129), (300, 300)])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(nq, nk, causal):
    dense(1, nq, nk, 2, 1, 64, causal=causal, seed=nq)


@pytest.mark.parametrize("d", [8, 24, 32, 40, 64, 72, 96, 104, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_head_widths(d, dtype):
    dense(1, 150, 170, 2, 2, d, dtype=dtype, causal=True, seed=d)


@pytest.mark.parametrize("heads,kv,batch", [(1, 1, 1), (8, 1, 1), (6, 3, 2), (8, 8, 2), (16, 4, 1)])
def test_head_groups(heads, kv, batch):
    dense(batch, 100, 100, heads, kv, 64, causal=True, seed=heads)


@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 1000])
def test_windows(window):
    dense(1, 260, 260, 2, 1, 64, causal=True, window=window, seed=window)
    dense(1, 130, 300, 2, 1, 128, causal=True, window=window, seed=window)


@pytest.mark.parametrize("nq,nk,causal,window", [(1, 1, True, 0), (130, 1, False, 0), (200, 200, True, 1), (40, 300, True, 1)])
@pytest.mark.parametrize("d", [32, 64, 88, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_visible_key_has_no_score_gradient(nq, nk, causal, window, d, dtype):
    """softmax over one key is 1 whatever the score: dq and dk are zero, not round-off, and out is the value."""
    torch = _torch()
    print(f"attention one key {nq} {nk} {d} {dtype}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(nq + d)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(_dt(dtype))  # noqa: E731
    q, k, v, dout = mk(2, nq, 4, d), mk(2, nk, 2, d), mk(2, nk, 2, d), mk(2, nq, 4, d)
    got = run(q, k, v, dout, causal=causal, window=window)
    j = torch.arange(nq, device="cuda") + nk - nq if causal else torch.zeros(nq, dtype=torch.int64, device="cuda")
    assert torch.equal(got["out"], v[:, j].repeat_interleave(2, dim=2))
    assert (got["dq"] == 0).all() and (got["dk"] == 0).all()


def test_large_scores_and_scales():
    dense(1, 200, 200, 2, 1, 128, spread=30.0, seed=1)
    dense(1, 200, 200, 2, 1, 64, scale=1.0, seed=2)
    dense(1, 200, 200, 2, 1, 64, scale=1e-3, seed=3)


def test_longer_than_one_workgroup():
    dense(1, 1100, 1100, 2, 1, 128, causal=True, seed=5)


@pytest.mark.parametrize("nq,nk,causal,window", [(1, 3000, False, 0), (1, 1025, True, 0), (100, 5000, True, 0), (129, 4100, True, 1500),
                                                (7, 9000, False, 0), (600, 2000, False, 0), (40, 2000, True, 30)])
@pytest.mark.parametrize("d", [64, 128, 72])
def test_few_queries_on_a_long_context(nq, nk, causal, window, d):
    """The keys of these are split over workgroups and joined."""
    dense(1, nq, nk, 2, 1, d, causal=causal, window=window, seed=nq + d)


@pytest.mark.parametrize("batch,heads,kv,causal", [(16, 16, 8, False), (32, 32, 32, True), (3, 5, 5, True)])
def test_many_workgroups(batch, heads, kv, causal):
    """Launches of many even and uneven workgroups, and a head count that does not spread over eight."""
    dense(batch, 200, 200, heads, kv, 64, causal=causal, seed=batch)


def test_packed_sequences_on_long_contexts():
    torch = _torch()
    print("attention packed long", flush=True)
    nq, nk = [3, 0, 90, 1], [4000, 50, 100, 2000]
    mk = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    q, k, v, dout = mk(sum(nq), 2, 128), mk(sum(nk), 1, 128), mk(sum(nk), 1, 128), mk(sum(nq), 2, 128)
    st = lambda n: torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")  # noqa: E731
    got = run(q, k, v, dout, causal=True, q_start=st(nq), k_start=st(nk), max_q=max(nq), max_k=max(nk))
    got = {n: np64(t) for n, t in got.items()}
    a = c = 0
    for m, n in zip(nq, nk):
        one = {x: got[x][a:a + m] for x in ("out", "dq")} | {x: got[x][c:c + n] for x in ("dk", "dv")}
        one["lse"] = got["lse"][:, a:a + m]
        check_sequence(np64(q[a:a + m]), np64(k[c:c + n]), np64(v[c:c + n]), np64(dout[a:a + m]), one, 128 ** -0.5,
                       T.visible(m, n, True), U["bf16"])
        a, c = a + m, c + n


@pytest.mark.parametrize("count", [64, 65, 200, 256, 300])
def test_many_packed_sequences(count):
    """More sequences than a wavefront has lanes, and than the list of blocks takes."""
    torch = _torch()
    print(f"attention packed {count}", flush=True)
    rng = np.random.default_rng(count)
    lens = [int(x) for x in rng.integers(0, 9, count)]
    lens[count // 2], lens[-1], lens[3] = 300, 140, 0
    mk = lambda h: torch.randn(sum(lens), h, 32, device="cuda").bfloat16()  # noqa: E731
    q, k, v, dout = mk(2), mk(1), mk(1), mk(2)
    st = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    for causal in (True, False):
        got = {n: np64(t) for n, t in run(q, k, v, dout, causal=causal, q_start=st, k_start=st, max_q=300, max_k=300).items()}
        a = 0
        for m in lens:
            one = {x: got[x][a:a + m] for x in ("out", "dq", "dk", "dv")} | {"lse": got["lse"][:, a:a + m]}
            if m:
                check_sequence(np64(q[a:a + m]), np64(k[a:a + m]), np64(v[a:a + m]), np64(dout[a:a + m]), one, 32 ** -0.5,
                               T.visible(m, m, causal), U["bf16"])
            a += m


def test_rising_scores_move_the_running_maximum():
    """Keys whose scores grow along the sequence raise the maximum in every tile."""
    torch = _torch()
    print("attention rising", flush=True)
    q = torch.ones(1, 40, 1, 64, device="cuda").bfloat16()
    k = torch.linspace(-3, 3, 700, device="cuda")[None, :, None, None].expand(1, 700, 1, 64).bfloat16()
    v = torch.randn(1, 700, 1, 64, device="cuda").bfloat16()
    got = {n: np64(t) for n, t in run(q, k, v, q, scale=1.0).items()}
    check_sequence(np64(q[0]), np64(k[0]), np64(v[0]), np64(q[0]), {n: got[n][0] for n in ("out", "dq", "dk", "dv")} |
                   {"lse": got["lse"]}, 1.0, T.visible(40, 700), U["bf16"])


@pytest.mark.parametrize("lens", [([5], [5]), ([1, 130, 0, 64, 7], [1, 130, 0, 64, 7]),
                                  ([100, 3, 200], [40, 90, 200]), ([0, 10], [7, 0])])
@pytest.mark.parametrize("window", [0, 9])
def test_packed_sequences(lens, window):
    torch = _torch()
    print(f"attention packed {lens} {window}", flush=True)
    nq, nk = lens
    g = torch.Generator(device="cuda").manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v, dout = mk(sum(nq), 4, 64), mk(sum(nk), 2, 64), mk(sum(nk), 2, 64), mk(sum(nq), 4, 64)
    st = lambda n: torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")  # noqa: E731
    got = run(q, k, v, dout, causal=True, window=window, q_start=st(nq), k_start=st(nk), max_q=max(nq), max_k=max(nk))
    got = {n: np64(t) for n, t in got.items()}
    a = c = 0
    for m, n in zip(nq, nk):
        one = {x: got[x][a:a + m] for x in ("out", "dq")} | {x: got[x][c:c + n] for x in ("dk", "dv")}
        one["lse"] = got["lse"][:, a:a + m]
        if m or n:
            check_sequence(np64(q[a:a + m]), np64(k[c:c + n]), np64(v[c:c + n]), np64(dout[a:a + m]), one, 0.125,
                           T.visible(m, n, True, window), U["bf16"])
        a, c = a + m, c + n


@pytest.mark.parametrize("causal", [False, True])
def test_padding_is_never_read(causal):
    """Past each length every input holds NaN; outputs and gradients there are zeros."""
    torch = _torch()
    print("attention padded", causal, flush=True)
    g = torch.Generator(device="cuda").manual_seed(4)
    lens_q, lens_k = [0, 70, 200, 131], [9, 200, 1, 131]
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v, dout = mk(4, 200, 2, 64), mk(4, 200, 1, 64), mk(4, 200, 1, 64), mk(4, 200, 2, 64)
    for b in range(4):
        q[b, lens_q[b]:], dout[b, lens_q[b]:] = float("nan"), float("nan")
        k[b, lens_k[b]:], v[b, lens_k[b]:] = float("nan"), float("inf")
    ti = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = {n: np64(t) for n, t in run(q, k, v, dout, causal=causal, q_lens=ti(lens_q), k_lens=ti(lens_k)).items()}
    lse = got["lse"].reshape(2, 4, 200)
    for b, (m, n) in enumerate(zip(lens_q, lens_k)):
        for x, e in (("out", m), ("dq", m), ("dk", n), ("dv", n)):
            assert (got[x][b, e:] == 0).all(), x
        assert np.isneginf(lse[:, b, m:]).all()
        if m:
            one = {x: got[x][b, :m] for x in ("out", "dq")} | {x: got[x][b, :n] for x in ("dk", "dv")}
            check_sequence(np64(q[b, :m]), np64(k[b, :n]), np64(v[b, :n]), np64(dout[b, :m]),
                           one | {"lse": lse[:, b, :m]}, 0.125, T.visible(m, n, causal), U["bf16"])
        else:
            assert (got["dk"][b] == 0).all() and (got["dv"][b] == 0).all()


@pytest.mark.parametrize("tokens", [1, 2])   # 1: one workgroup's rows; 2: workgroups of two sets and splits
def test_rows_and_keys_that_see_nothing_among_values_that_are_not_finite(tokens):
    """Rows without a key, queries past their length and keys without a query
    share tiles with values that are not finite."""
    torch, train = _torch(), _train()
    print("attention nothing visible", tokens, flush=True)
    g = torch.Generator(device="cuda").manual_seed(14)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    ti = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    nk = 8 if tokens == 1 else 700
    nq = nk + 40                       # causal: the first 40 queries see no key
    q, k, v, dout = mk(1, nq, 2, 64), mk(1, nk, 1, 64), mk(1, nk, 1, 64), mk(1, nq, 2, 64)
    k[:, ::3], v[:, ::2] = float("nan"), float("inf")
    got = run(q, k, v, dout, causal=True)
    assert not got["out"][:, :40].any() and not got["dq"][:, :40].any()
    assert got["lse"][:, :40].isneginf().all()
    lens = [30, 0]                     # not causal: queries past 30 are padding, and a whole sequence of them
    q, k, v, dout = mk(2, 60, 2, 64), mk(2, nk, 1, 64), mk(2, nk, 1, 64), mk(2, 60, 2, 64)
    k[:, ::3], v[:, ::2] = float("inf"), float("nan")
    got = run(q, k, v, dout, q_lens=ti(lens))
    for b, n in enumerate(lens):
        assert not got["out"][b, n:].any() and not got["dq"][b, n:].any()
    q, k, v, dout = mk(1, 20, 2, 64), mk(1, nk + 60, 1, 64), mk(1, nk + 60, 1, 64), mk(1, 20, 2, 64)
    q[:, ::3], dout[:, ::2] = float("nan"), float("inf")
    out, lse = train.attention_forward(q, k, v, causal=True, window=4)   # the last 23 keys have queries
    _, dk, dv = train.attention_backward(dout, q, k, v, out, lse, causal=True, window=4)
    assert not dk[:, :-23].any() and not dv[:, :-23].any()


def test_more_workgroups_than_one_launch_holds():
    """Past 2^31 threads the row blocks take several launches. One token a
    sequence: its output is its value."""
    torch, train = _torch(), _train()
    batch, heads = 2 ** 17 + 3, 64
    print("attention workgroups", batch * heads, flush=True)
    g = torch.Generator(device="cuda").manual_seed(15)
    q, k, v, dout = (torch.randn(batch, 1, heads, 8, generator=g, device="cuda").bfloat16() for _ in range(4))
    out, lse = train.attention_forward(q, k, v, scale=0.25)
    dq, dk, dv = train.attention_backward(dout, q, k, v, out, lse, scale=0.25)
    assert torch.equal(out, v) and torch.equal(dv, dout) and not dq.any() and not dk.any()
    s = 0.25 * (q.double() * k.double()).sum(-1)[:, 0].t()
    # eight products of 24 bits added in 24, the scaling and the change of base: 16 roundings of the largest sum
    most = 0.25 * (q.double() * k.double()).abs().sum(-1)[:, 0].t()
    assert ((lse.reshape(heads, batch) - s).abs() <= 16 * 2.0 ** -24 * most + 1e-30).all()


def test_strided_views_and_given_outputs():
    """q, k, v are views of one projection, their gradients views of another, and out is head-major."""
    torch, train = _torch(), _train()
    print("attention strided", flush=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(2, 90, 8 * 64, generator=g, device="cuda").bfloat16()
    q, k, v = x.view(2, 90, 8, 64).split([4, 2, 2], dim=2)
    dx = torch.full_like(x, float("nan"))
    dq, dk, dv = dx.view(2, 90, 8, 64).split([4, 2, 2], dim=2)
    out = torch.empty(2, 4, 90, 64, device="cuda", dtype=torch.bfloat16).transpose(1, 2)
    dout = torch.randn(2, 4, 90, 64, generator=g, device="cuda").bfloat16().transpose(1, 2)
    o, lse = train.attention_forward(q, k, v, causal=True, out=out)
    r = train.attention_backward(dout, q, k, v, o, lse, causal=True, dq=dq, dk=dk, dv=dv)
    o2, lse2 = train.attention_forward(q.contiguous(), k.contiguous(), v.contiguous(), causal=True)
    r2 = train.attention_backward(dout.contiguous(), q.contiguous(), k.contiguous(), v.contiguous(), o2, lse2, causal=True)
    torch.cuda.synchronize()
    assert o is out and r[0] is dq
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(a, b) for a, b in zip(r, r2))
    assert not dx.isnan().any()


def test_expanded_gradient():
    """The gradient of a sum is an expanded scalar, with strides of 0."""
    torch, train = _torch(), _train()
    print("attention expanded", flush=True)
    q = torch.randn(1, 70, 2, 64, device="cuda").bfloat16()
    out, lse = train.attention_forward(q, q, q)
    one = torch.ones((), device="cuda", dtype=torch.bfloat16).expand(q.shape)
    a = train.attention_backward(one, q, q, q, out, lse)
    b = train.attention_backward(one.contiguous(), q, q, q, out, lse)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_expanded_gradient_on_another_stream():
    """The copy that an expanded gradient needs is made on the stream of the call."""
    torch, train = _torch(), _train()
    print("attention expanded, stream", flush=True)
    q = torch.randn(2, 1500, 4, 64, device="cuda").bfloat16()
    out, lse = train.attention_forward(q, q, q)
    one = torch.ones((), device="cuda", dtype=torch.bfloat16).expand(q.shape)
    want = train.attention_backward(one, q, q, q, out, lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(10):
        busy = busy @ busy / 64   # the current stream is not done when the call is made
    got = train.attention_backward(one, q, q, q, out, lse, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_windows_past_the_keys():
    dense(1, 70, 100, 2, 1, 64, causal=True, window=100, seed=8)
    torch, train = _torch(), _train()
    q = torch.randn(1, 90, 1, 64, device="cuda").bfloat16()
    assert torch.equal(train.attention_forward(q, q, q, causal=True, window=2 ** 31 - 1)[0],
                       train.attention_forward(q, q, q, causal=True)[0])


def test_bad_offsets_stay_inside():
    """Offsets that descend or leave the token axis give defined, in-bounds work: no row outside is written."""
    torch, train = _torch(), _train()
    print("attention offsets", flush=True)
    x = torch.randn(60, 2, 64, device="cuda").bfloat16()
    st = torch.tensor([0, 50, 20, 1000], dtype=torch.int32, device="cuda")
    buf = torch.full((100, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    out, lse = train.attention_forward(x, x, x, causal=True, q_start=st, k_start=st, max_q=64, max_k=64, out=buf[20:80])
    torch.cuda.synchronize()
    assert (buf[:20] == 7).all() and (buf[80:] == 7).all()


def test_empty_calls():
    torch, train = _torch(), _train()
    print("attention empty", flush=True)
    q, k = torch.zeros(2, 0, 2, 64, device="cuda").bfloat16(), torch.zeros(2, 5, 2, 64, device="cuda").bfloat16()
    out, lse = train.attention_forward(q, k, k)
    assert out.shape == q.shape and lse.shape == (2, 0)
    dq, dk, dv = train.attention_backward(q, q, k, k, out, lse)
    assert (dk == 0).all() and (dv == 0).all()
    out, lse = train.attention_forward(k, q, q)
    assert (out == 0).all() and torch.isneginf(lse).all()
    dq, dk, dv = train.attention_backward(k, k, q, q, out, lse)
    assert (dq == 0).all() and dk.shape == q.shape


def test_nan_and_infinity_reach_their_rows():
    torch, train = _torch(), _train()
    print("attention nan", flush=True)
    q, k = torch.randn(1, 130, 1, 64, device="cuda").bfloat16(), torch.randn(1, 130, 1, 64, device="cuda").bfloat16()
    q[0, 70] = float("nan")
    out, lse = train.attention_forward(q, k, k, causal=True)
    rows = out[0, :, 0].isnan().any(dim=1)
    assert rows[70] and rows.sum() == 1 and lse[0].isnan().sum() == 1


def test_equal_bits_on_another_stream_and_in_a_graph():
    torch, train = _torch(), _train()
    print("attention streams", flush=True)
    q = torch.randn(2, 300, 4, 128, device="cuda").bfloat16()
    k = torch.randn(2, 300, 2, 128, device="cuda").bfloat16()
    first = run(q, k, k, q, causal=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = train.attention_forward(q, k, k, causal=True, stream=s)
    grads = train.attention_backward(q, q, k, k, out, lse, causal=True, stream=s)
    s.synchronize()
    want = [first[n] for n in ("out", "lse", "dq", "dk", "dv")]
    assert all(torch.equal(a, b) for a, b in zip((out, lse, *grads), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = train.attention_forward(q, k, k, causal=True)
        grads = train.attention_backward(q, q, k, k, out, lse, causal=True)
    for n in range(3):
        q.copy_(torch.randn_like(q))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, lse, *grads)]
        again = run(q, k, k, q, causal=True)
        assert all(torch.equal(a, again[n]) for a, n in zip(got, ("out", "lse", "dq", "dk", "dv"))), n


def test_equal_bits_with_wavefronts_that_skip_tiles():
    """Packed causal sequences, where a workgroup's wavefronts skip different
    tiles but copy their share of each: a launch must give the same bits among
    other launches on other data."""
    torch = _torch()
    print("attention repeated", flush=True)
    lens = [700, 45, 1, 130, 260, 33, 1100, 64]
    st = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    how = dict(causal=True, q_start=st, k_start=st, max_q=max(lens), max_k=max(lens))
    mk = lambda h: torch.randn(sum(lens), h, 128, device="cuda").bfloat16()  # noqa: E731
    sets = [(mk(8), mk(4), mk(4), mk(8)) for _ in range(2)]
    first = [run(*s, **how) for s in sets]
    for n in range(6):
        got = [run(*s, **how) for s in sets + sets]
        for a, b in zip(got, first + first):
            assert all(torch.equal(a[x], b[x]) for x in a), n
    c = {n: np64(t) for n, t in first[0].items()}
    q, k, v, dout = (np64(t) for t in sets[0])
    a = 0
    for m in lens:
        one = {x: c[x][a:a + m] for x in ("out", "dq", "dk", "dv")} | {"lse": c["lse"][:, a:a + m]}
        check_sequence(q[a:a + m], k[a:a + m], v[a:a + m], dout[a:a + m], one, 128 ** -0.5, T.visible(m, m, True), U["bf16"])
        a += m


@pytest.mark.parametrize("window", [0, 5])
@pytest.mark.parametrize("case", ["gaps", "cut", "no sequences", "no lengths"])
def test_packed_tokens_outside_every_sequence_are_zeros(case, window):
    """Before the first sequence, after the last one and past max_q or max_k: outputs and gradients 0, lse -inf, in
    memory that held NaN before."""
    torch, train = _torch(), _train()
    print(f"attention packed, uncovered {case} {window}", flush=True)
    ti = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    nq, nk, h, hk, d = 700, 900, 4, 2, 64
    qs, ks, mq, mk_ = {"gaps": ([3, 3, 200, 650], [100, 130, 400, 890], 450, 490),
                       "cut": ([0, 300, 300, 700], [0, 20, 500, 900], 130, 70),
                       "no sequences": ([0], [0], 10, 10), "no lengths": ([0, 700], [0, 900], 0, 0)}[case]
    g = torch.Generator(device="cuda").manual_seed(16)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v, dout = mk(nq, h, d), mk(nk, hk, d), mk(nk, hk, d), mk(nq, h, d)
    cover = lambda s, most, n: [(a, min(max(b, a), a + most)) for a, b in zip(s[:-1], s[1:])]  # noqa: E731
    cq, ck = cover(qs, mq, nq), cover(ks, mk_, nk)
    for t, c in ((q, cq), (dout, cq), (k, ck), (v, ck)):   # never read either
        keep = torch.zeros(len(t), dtype=torch.bool, device="cuda")
        for a, b in c:
            keep[a:b] = True
        t[~keep] = float("nan")
    how = dict(causal=True, window=window, q_start=ti(qs), k_start=ti(ks), max_q=mq, max_k=mk_)
    bad = lambda like: torch.full_like(like, float("nan"))  # noqa: E731
    for given in (False, True):
        held = [bad(q) for _ in range(6)] + [bad(k) for _ in range(4)] + [torch.full((h, nq), float("nan"), device="cuda")]
        del held
        out, lse = train.attention_forward(q, k, v, out=bad(q) if given else None, **how)
        more = dict(dq=bad(q), dk=bad(k), dv=bad(k)) if given else {}
        dq, dk, dv = train.attention_backward(dout, q, k, v, out, lse, **how, **more)
        got = {n: np64(t) for n, t in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv))}
        for (a, m), (c, n) in zip(cq, ck):
            one = {x: got[x][a:m] for x in ("out", "dq")} | {x: got[x][c:n] for x in ("dk", "dv")}
            check_sequence(np64(q[a:m]), np64(k[c:n]), np64(v[c:n]), np64(dout[a:m]), one | {"lse": got["lse"][:, a:m]},
                           d ** -0.5, T.visible(m - a, n - c, True, window), U["bf16"])
            got["out"][a:m], got["dq"][a:m], got["lse"][:, a:m] = 0, 0, -np.inf
            got["dk"][c:n], got["dv"][c:n] = 0, 0
        for x in ("out", "dq", "dk", "dv"):
            assert (got[x] == 0).all(), x
        assert np.isneginf(got["lse"]).all()


def test_half_precision_value_gradients_over_many_keys():
    """Each of n keys that are seen alike has the probability 1 / n: far below float16's normal numbers, and no less
    exact. dv_j = dout / n is off by the two roundings, u each, and the fp32 arithmetic's 2^-12."""
    torch, train = _torch(), _train()
    n = 10 ** 6
    print("attention f16, keys", n, flush=True)
    g = torch.Generator(device="cuda").manual_seed(17)
    q = torch.zeros(1, 1, 1, 64, device="cuda").half()
    k, v = (torch.randn(1, n, 1, 64, generator=g, device="cuda").half() for _ in range(2))
    dout = (1000 * (1 + torch.rand(1, 1, 1, 64, generator=g, device="cuda"))).half()
    out, lse = train.attention_forward(q, k, v)
    dq, dk, dv = train.attention_backward(dout, q, k, v, out, lse)
    want = dout.double() / n   # above 2^-14 everywhere
    assert ((dv.double() - want).abs() <= (2 * U["f16"] + SLACK) * want).all()


@pytest.mark.parametrize("nq,nk,causal", [(3000, 100, False), (2000, 130, True), (100, 4000, True)])
@pytest.mark.parametrize("d", [64, 128])
def test_half_precision_over_splits(nq, nk, causal, d):
    """Queries (or keys) split over workgroups, whose fp32 parts a second kernel joins."""
    dense(1, nq, nk, 2, 1, d, dtype="f16", causal=causal, seed=nq + d)


def some(batch, heads, kv, d, dtype, causal, n=300, pick=3):
    """Like dense, but only a few of the sequences are compared."""
    torch = _torch()
    print(f"attention {batch}x{n} heads {heads}/{kv} d {d} {dtype} causal {causal}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(d + batch)
    mk = lambda h: torch.randn(batch, n, h, d, generator=g, device="cuda").to(_dt(dtype))  # noqa: E731
    q, k, v, dout = mk(heads), mk(kv), mk(kv), mk(heads)
    got = run(q, k, v, dout, causal=causal)
    lse = got["lse"].view(heads, batch, n)
    for b in sorted({0, batch // 2, batch - 1})[:pick]:
        one = {x: np64(got[x][b]) for x in ("out", "dq", "dk", "dv")} | {"lse": np64(lse[:, b])}
        check_sequence(np64(q[b]), np64(k[b]), np64(v[b]), np64(dout[b]), one, d ** -0.5, T.visible(n, n, causal), U[dtype])
    assert all(t.isfinite().all() for t in got.values())


# Blocks of 128 rows times heads: up to 256 take two sets of wavefronts, below 1024 one set of four, from there eight
@pytest.mark.parametrize("batch,heads,kv", [(7, 16, 16), (14, 16, 8), (22, 16, 16), (43, 16, 8)])
@pytest.mark.parametrize("d", [72, 96, 128])
@pytest.mark.parametrize("dtype,causal", [("bf16", True), ("bf16", False), ("f16", True), ("f16", False)])
def test_wide_heads_in_every_workgroup_shape(batch, heads, kv, d, dtype, causal):
    """Forward, dQ and dK/dV of 300 tokens (a ragged tail in each shape's last block): 336 and 672 blocks, 1056 and 2064."""
    some(batch, heads, kv, d, dtype, causal)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,count", [(96, 60), (128, 60), (128, 300)])
def test_wide_heads_of_many_packed_sequences(d, count, dtype):
    """Enough packed blocks for eight wavefronts a workgroup, found in the list and (past 256 sequences) without it."""
    torch = _torch()
    print(f"attention packed wide {d} {count} {dtype}", flush=True)
    rng = np.random.default_rng(count + d)
    lens = [int(x) for x in rng.integers(0, 300 if count == 60 else 60, count)]
    lens[1], lens[count // 2], lens[-1] = 0, 517, 1
    g = torch.Generator(device="cuda").manual_seed(count)
    mk = lambda h: torch.randn(sum(lens), h, d, generator=g, device="cuda").to(_dt(dtype))  # noqa: E731
    q, k, v, dout = mk(16), mk(16), mk(16), mk(16)
    at = np.concatenate([[0], np.cumsum(lens)])
    st = torch.tensor(at, dtype=torch.int32, device="cuda")
    got = run(q, k, v, dout, causal=True, q_start=st, k_start=st, max_q=517, max_k=517)
    assert all(t.isfinite().all() for t in got.values())
    for b in (0, 1, 2, count // 2, count - 1):
        a, e = int(at[b]), int(at[b + 1])
        if e > a:
            one = {x: np64(got[x][a:e]) for x in ("out", "dq", "dk", "dv")} | {"lse": np64(got["lse"][:, a:e])}
            check_sequence(np64(q[a:e]), np64(k[a:e]), np64(v[a:e]), np64(dout[a:e]), one, d ** -0.5,
                           T.visible(e - a, e - a, True), U[dtype])
