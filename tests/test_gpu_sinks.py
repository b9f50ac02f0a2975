"""GPU tests of attention with a sliding window and first keys that stay visible
(sinks), against the fp64 oracle with the bounds of test_gpu_attention.py."""

import numpy as np
import pytest

from oracle import train_ops as T
from tests.test_gpu_attention import U, check_sequence, np64, run

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _train():
    from matrix_optimizer_step_02_amd import train
    return train


def _dt(name):
    torch = _torch()
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def normal(seed, dtype="bf16"):
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda").to(_dt(dtype))


def dense(batch, nq, nk, heads, kv, d, window, sinks, dtype="bf16", seed=0, forward=False):
    print(f"sinks {batch}x{nq}x{nk} heads {heads}/{kv} d {d} window {window} sinks {sinks} {dtype}", flush=True)
    mk = normal(seed, dtype)
    q, k, v, dout = mk(batch, nq, heads, d), mk(batch, nk, kv, d), mk(batch, nk, kv, d), mk(batch, nq, heads, d)
    got = run(q, k, v, None if forward else dout, causal=True, window=window, sinks=sinks)
    got = {n: np64(t) for n, t in got.items()}
    see = T.visible(nq, nk, True, window, sinks)
    lse = got["lse"].reshape(heads, batch, nq)
    for b in range(batch):
        one = {n: got[n][b] for n in ("out", "dq", "dk", "dv") if n in got} | {"lse": lse[:, b]}
        check_sequence(np64(q[b]), np64(k[b]), np64(v[b]), None if forward else np64(dout[b]), one, d ** -0.5, see, U[dtype])


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 100, 128, 300])
@pytest.mark.parametrize("sinks", [1, 4, 63, 64, 65, 127, 130, 500])
def test_windows_and_sinks(window, sinks):
    dense(1, 420, 420, 2, 1, 64, window, sinks, seed=window + sinks)


@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 2), (1, 64), (1, 700), (2, 300), (31, 33), (64, 64), (129, 200), (200, 129), (300, 5),
                                   (5, 300), (130, 900)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (5, 3), (70, 4), (40, 70)])
def test_lengths(nq, nk, window, sinks):
    dense(1, nq, nk, 2, 1, 128, window, sinks, seed=nq + nk)


@pytest.mark.parametrize("d", [8, 32, 40, 64, 72, 96, 104, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("batch", [1, 24])
def test_widths_and_shapes(d, dtype, batch):
    """Few and many workgroups: each of their shapes."""
    dense(batch, 330, 330, 4, 2, d, 50, 9, dtype=dtype, seed=d)


@pytest.mark.parametrize("heads,kv,batch", [(1, 1, 1), (8, 1, 1), (6, 3, 2), (8, 8, 2), (16, 4, 3)])
def test_head_groups(heads, kv, batch):
    dense(batch, 190, 190, heads, kv, 64, 33, 4, seed=heads)


@pytest.mark.parametrize("nq,nk,window,sinks", [(1, 5000, 1000, 4), (3, 9000, 8000, 4), (100, 5000, 700, 130), (600, 3000, 2000, 4),
                                                (1, 3000, 5, 1000), (2100, 2100, 64, 4), (2100, 2100, 1500, 300)])
@pytest.mark.parametrize("d", [64, 128])
def test_long_contexts(nq, nk, window, sinks, d):
    """Keys of a query and queries of the sinks that are split over workgroups and joined."""
    dense(1, nq, nk, 2, 1, d, window, sinks, seed=nq + d)


@pytest.mark.parametrize("heads,kv,batch,d", [(16, 8, 3, 128), (16, 4, 5, 64), (4, 4, 16, 96), (8, 1, 40, 32)])
def test_single_tokens(heads, kv, batch, d):
    """One query a sequence on caches of uneven lengths; NaN past each."""
    torch = _torch()
    print(f"sinks one token {heads}/{kv} batch {batch} d {d}", flush=True)
    mk = normal(d)
    r = np.random.default_rng(batch)
    nk = [1, 2, 70] + [int(x) for x in r.integers(1, 2500, batch - 3)]
    most = max(nk)
    q, k, v, dout = mk(batch, 1, heads, d), mk(batch, most, kv, d), mk(batch, most, kv, d), mk(batch, 1, heads, d)
    for b, n in enumerate(nk):
        k[b, n:], v[b, n:] = float("nan"), float("inf")
    lens = torch.tensor(nk, dtype=torch.int32, device="cuda")
    got = {n: np64(t) for n, t in run(q, k, v, dout, causal=True, window=200, sinks=4, k_lens=lens).items()}
    lse = got["lse"].reshape(heads, batch, 1)
    for b, n in enumerate(nk):
        assert not got["dk"][b, n:].any() and not got["dv"][b, n:].any()
        one = {x: got[x][b] for x in ("out", "dq")} | {x: got[x][b, :n] for x in ("dk", "dv")} | {"lse": lse[:, b]}
        check_sequence(np64(q[b]), np64(k[b, :n]), np64(v[b, :n]), np64(dout[b]), one, d ** -0.5,
                       T.visible(1, n, True, 200, 4), U["bf16"])


@pytest.mark.parametrize("lens", [([5], [5]), ([1, 130, 0, 64, 7], [1, 130, 0, 64, 7]), ([100, 3, 200], [40, 90, 200]),
                                  ([0, 10], [7, 0]), ([700, 1, 300], [700, 1, 300])])
@pytest.mark.parametrize("window,sinks", [(9, 4), (64, 70), (1, 1)])
def test_packed_sequences(lens, window, sinks):
    """Uncovered tokens before, between and behind the sequences come back as zeros."""
    torch = _torch()
    print(f"sinks packed {lens} {window} {sinks}", flush=True)
    nq, nk = lens
    mk = normal(3)
    q, k, v, dout = mk(sum(nq) + 5, 4, 64), mk(sum(nk) + 5, 2, 64), mk(sum(nk) + 5, 2, 64), mk(sum(nq) + 5, 4, 64)
    st = lambda n: torch.tensor(3 + np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")  # noqa: E731
    got = run(q, k, v, dout, causal=True, window=window, sinks=sinks, q_start=st(nq), k_start=st(nk), max_q=max(nq), max_k=max(nk))
    got = {n: np64(t) for n, t in got.items()}
    a = c = 3
    for m, n in zip(nq, nk):
        one = {x: got[x][a:a + m] for x in ("out", "dq")} | {x: got[x][c:c + n] for x in ("dk", "dv")}
        one["lse"] = got["lse"][:, a:a + m]
        if m or n:
            check_sequence(np64(q[a:a + m]), np64(k[c:c + n]), np64(v[c:c + n]), np64(dout[a:a + m]), one, 0.125,
                           T.visible(m, n, True, window, sinks), U["bf16"])
        a, c = a + m, c + n
    for x in ("out", "dq", "dk", "dv"):
        assert not got[x][:3].any() and not got[x][-2:].any(), x


@pytest.mark.parametrize("count", [65, 300])
def test_many_packed_sequences(count):
    torch = _torch()
    print(f"sinks packed {count}", flush=True)
    rng = np.random.default_rng(count)
    lens = [int(x) for x in rng.integers(0, 9, count)]
    lens[count // 2], lens[-1], lens[3] = 300, 140, 0
    mk = normal(count)
    n = sum(lens)
    q, k, v, dout = mk(n, 2, 32), mk(n, 1, 32), mk(n, 1, 32), mk(n, 2, 32)
    st = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    got = {x: np64(t) for x, t in run(q, k, v, dout, causal=True, window=20, sinks=6, q_start=st, k_start=st, max_q=300,
                                      max_k=300).items()}
    a = 0
    for m in lens:
        one = {x: got[x][a:a + m] for x in ("out", "dq", "dk", "dv")} | {"lse": got["lse"][:, a:a + m]}
        if m:
            check_sequence(np64(q[a:a + m]), np64(k[a:a + m]), np64(v[a:a + m]), np64(dout[a:a + m]), one, 32 ** -0.5,
                           T.visible(m, m, True, 20, 6), U["bf16"])
        a += m


def test_padding_is_never_read():
    torch = _torch()
    print("sinks padded", flush=True)
    lens_q, lens_k = [0, 70, 200, 131, 200], [9, 200, 1, 131, 200]
    mk = normal(4)
    q, k, v, dout = mk(5, 200, 2, 64), mk(5, 200, 1, 64), mk(5, 200, 1, 64), mk(5, 200, 2, 64)
    for b in range(5):
        q[b, lens_q[b]:], dout[b, lens_q[b]:] = float("nan"), float("nan")
        k[b, lens_k[b]:], v[b, lens_k[b]:] = float("nan"), float("inf")
    ti = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = run(q, k, v, dout, causal=True, window=30, sinks=70, q_lens=ti(lens_q), k_lens=ti(lens_k))
    got = {n: np64(t) for n, t in got.items()}
    lse = got["lse"].reshape(2, 5, 200)
    for b, (m, n) in enumerate(zip(lens_q, lens_k)):
        for x, e in (("out", m), ("dq", m), ("dk", n), ("dv", n)):
            assert (got[x][b, e:] == 0).all(), x
        assert np.isneginf(lse[:, b, m:]).all()
        if m:
            one = {x: got[x][b, :m] for x in ("out", "dq")} | {x: got[x][b, :n] for x in ("dk", "dv")}
            check_sequence(np64(q[b, :m]), np64(k[b, :n]), np64(v[b, :n]), np64(dout[b, :m]),
                           one | {"lse": lse[:, b, :m]}, 0.125, T.visible(m, n, True, 30, 70), U["bf16"])


def test_rows_that_see_nothing_among_values_that_are_not_finite():
    """The first 40 queries come before every key; keys between the sinks and the window have no query."""
    torch, train = _torch(), _train()
    print("sinks nothing visible", flush=True)
    mk = normal(14)
    q, k, v, dout = mk(1, 740, 2, 64), mk(1, 700, 1, 64), mk(1, 700, 1, 64), mk(1, 740, 2, 64)
    k[:, ::3], v[:, ::2] = float("nan"), float("inf")
    got = run(q, k, v, dout, causal=True, window=50, sinks=4)
    assert not got["out"][:, :40].any() and not got["dq"][:, :40].any()
    assert got["lse"][:, :40].isneginf().all()
    q, k, v, dout = mk(1, 20, 2, 64), mk(1, 700, 1, 64), mk(1, 700, 1, 64), mk(1, 20, 2, 64)
    q[:, ::3], dout[:, ::2] = float("nan"), float("inf")
    out, lse = train.attention_forward(q, k, v, causal=True, window=4, sinks=5)
    _, dk, dv = train.attention_backward(dout, q, k, v, out, lse, causal=True, window=4, sinks=5)
    assert not dk[:, 5:-23].any() and not dv[:, 5:-23].any()
    assert dk[:, :5].isnan().any()


def test_sinks_that_cover_everything_are_no_window():
    """Sinks as long as the keys, or a window as long, hide nothing: the same as causal attention within its rounding."""
    torch = _torch()
    mk = normal(6)
    q, k, v, dout = mk(2, 300, 4, 64), mk(2, 300, 2, 64), mk(2, 300, 2, 64), mk(2, 300, 4, 64)
    see = T.visible(300, 300, True)
    for window, sinks in ((10, 300), (10, 1 << 30), (10, 299), (300, 4), (1 << 30, 1), (299, 1)):
        got = {n: np64(t) for n, t in run(q, k, v, dout, causal=True, window=window, sinks=sinks).items()}
        lse = got["lse"].reshape(4, 2, 300)
        for b in range(2):
            one = {n: got[n][b] for n in ("out", "dq", "dk", "dv")} | {"lse": lse[:, b]}
            check_sequence(np64(q[b]), np64(k[b]), np64(v[b]), np64(dout[b]), one, 0.125, see, U["bf16"])


def test_no_sinks_is_the_window_to_the_bit():
    torch = _torch()
    mk = normal(7)
    q, k, v, dout = mk(1, 500, 4, 64), mk(1, 500, 2, 64), mk(1, 500, 2, 64), mk(1, 500, 4, 64)
    a = run(q, k, v, dout, causal=True, window=77)
    b = run(q, k, v, dout, causal=True, window=77, sinks=0)
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("nq,nk", [(600, 600), (2, 3000), (2100, 2100)])
def test_equal_inputs_give_equal_bits_and_graphs_replay(nq, nk):
    torch, train = _torch(), _train()
    print("sinks in a graph", nq, nk, flush=True)
    mk = normal(8)
    q, k, v, dout = mk(1, nq, 4, 128), mk(1, nk, 2, 128), mk(1, nk, 2, 128), mk(1, nq, 4, 128)
    call = lambda: run_unsynced(train, q, k, v, dout, causal=True, window=100, sinks=4)  # noqa: E731
    first = call()
    assert all(torch.equal(a, b) for a, b in zip(first, call()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for n in range(3):
        q.copy_(normal(20 + n)(1, nq, 4, 128))
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), n


def run_unsynced(train, q, k, v, dout, **how):
    out, lse = train.attention_forward(q, k, v, **how)
    return (out, lse, *train.attention_backward(dout, q, k, v, out, lse, **how))


@pytest.mark.parametrize("nq,nk,window,sinks,batch", [(1, 300, 4, 1, 2), (1, 300, 1, 3, 1), (2, 2, 22, 4, 3), (200, 200, 3, 2, 1),
                                                      (60, 60, 100, 4, 2), (300, 300, 2, 20, 1), (25, 25, 9, 9, 40)])
@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_of_few_keys_lose_nothing_to_rounded_outputs(nq, nk, window, sinks, batch, d, dtype):
    """Where a row sees few keys, D comes from P and dP in fp32 and not from the stored out: the bound of
    test_gpu_attention.py without out's error in D, which is off by what P and dP are, 2^-12 of sum P |dP|."""
    from tests.test_gpu_attention import SLACK, TINY, worst
    print(f"sinks few keys {nq} {nk} window {window} sinks {sinks} batch {batch} d {d} {dtype}", flush=True)
    mk = normal(nq + d, dtype)
    q, k, v, dout = mk(batch, nq, 4, d), mk(batch, nk, 2, d), mk(batch, nk, 2, d), mk(batch, nq, 4, d)
    got = {n: np64(t) for n, t in run(q, k, v, dout, causal=True, window=window, sinks=sinks).items()}
    see, u, scale = T.visible(nq, nk, True, window, sinks), U[dtype], d ** -0.5
    few = see.sum(1) < 32
    assert few.any()
    for b in range(batch):
        dk, bound = np.zeros((nk, 2, d)), np.zeros((nk, 2, d))
        for h in range(4):
            x, kk, vv, g = np64(q[b, :, h]), np64(k[b, :, h // 2]), np64(v[b, :, h // 2]), np64(dout[b, :, h])
            r = T.attention(x, kk, vv, scale, see, g)
            e_D = SLACK * (r["p"] * np.abs(r["dp"])).sum(1)
            e_ds = (u * np.abs(r["ds"]) + r["p"] * e_D[:, None] + SLACK * r["p"] * (np.abs(r["dp"]) + np.abs(r["D"])[:, None])
                    + TINY * see)
            e_dq = u * np.abs(r["dq"]) + scale * e_ds @ np.abs(kk) + SLACK * scale * np.abs(r["ds"]) @ np.abs(kk)
            assert worst(got["dq"][b, few, h], r["dq"][few], e_dq[few]) <= 1
            dk[:, h // 2] += r["dk"]
            bound[:, h // 2] += scale * e_ds.T @ np.abs(x) + SLACK * scale * np.abs(r["ds"]).T @ np.abs(x)
        if few.all():
            assert worst(got["dk"][b], dk, bound + u * np.abs(dk)) <= 1


def test_one_key_in_sight_has_no_score_gradient():
    """One query at the first position of a cache of one key, and windows of one key without other sinks in reach."""
    torch = _torch()
    mk = normal(3)
    for batch, nq, nk in ((17, 1, 1), (2, 40, 1)):
        q, k, v, dout = mk(batch, nq, 8, 64), mk(batch, nk, 4, 64), mk(batch, nk, 4, 64), mk(batch, nq, 8, 64)
        got = run(q, k, v, dout, causal=True, window=3, sinks=1)
        assert not got["dq"].any() and not got["dk"].any()
        assert torch.equal(got["out"][:, -1], v[:, 0].repeat_interleave(2, dim=1))


@pytest.mark.parametrize("nq", [1, 3])
def test_a_cache_past_2_31_elements(nq):
    """What lies between the sinks and the window is out of sight: without it the
    sequence gives the same."""
    torch, train = _torch(), _train()
    print(f"sinks cache past 2^31, {nq} queries", flush=True)
    batch, nk, heads, kv, d, window, sinks = 3, 700001, 16, 8, 128, 1000, 5
    tail = window + nq - 1
    mk = normal(nq)
    q, dout = mk(batch, nq, heads, d), mk(batch, nq, heads, d)
    k, v = (torch.zeros(batch, nk, kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 1 << 31
    seen = lambda t: torch.cat([t[:, :sinks], t[:, nk - tail:]], 1)  # noqa: E731
    for t in (k, v):
        t[:, :sinks] = mk(batch, sinks, kv, d)
        t[:, nk - tail:] = mk(batch, tail, kv, d)
    how = dict(causal=True, window=window, sinks=sinks)
    out, lse = train.attention_forward(q, k, v, **how)
    dq, dk, dv = train.attention_backward(dout, q, k, v, out, lse, **how)
    for t in (dk, dv):
        assert not bool(t[:, sinks:nk - tail].any())
    see = T.visible(nq, sinks + tail, True, window, sinks)
    ks, vs, dks, dvs = (np64(seen(t)) for t in (k, v, dk, dv))
    lse = np64(lse).reshape(heads, batch, nq)
    for b in range(batch):
        one = {"out": np64(out[b]), "dq": np64(dq[b]), "dk": dks[b], "dv": dvs[b], "lse": lse[:, b]}
        check_sequence(np64(q[b]), ks[b], vs[b], np64(dout[b]), one, d ** -0.5, see, U["bf16"])
