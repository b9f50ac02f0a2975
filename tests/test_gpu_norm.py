"""GPU tests of dropout and layer norm against the fp64 oracle.

Dropout is bitwise: mask, fp32 product, fp32 sum and rounding are defined.
Layer norm works in fp32 on the stored h: a sum of c terms in a tree of at
most 16 + 10 levels is off by 26 2^-24 of the sum of magnitudes, so mean, rstd
and the two gradient means are within 2^-19 of theirs, and with u = eps / 2 of
the output's type (0 slack for fp32 beyond the same 2^-18):
  y:  u |y| + 2^-18 (|xh w| + |b|)      dx: u |dx| + 2^-17 rstd (|z| + mean|z| + |xh| mean|z xh|) + 2^-23 |dh|
  dweight: (rows + 16) 2^-24 + 2^-19 of sum |dy xh|, with mean's own error 2^-19 rstd mean|h| sum |dy|
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


def _dt(name):
    torch = _torch()
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def np64(t):
    return t.detach().double().cpu().numpy()


def inside(got, ref, bound, what):
    r = float(np.max(np.abs(got - ref) / (bound + 1e-30))) if ref.size else 0.0
    assert r <= 1, f"{what}: {r}"


def dropped(x, p, seed, offset, res=None):
    """The operator's fp32 value of dropout(x) (+ res), before the last rounding."""
    torch = _torch()
    cols = x.shape[-1]
    f = T.dropout_factor(x.numel() // cols, cols, p, seed, offset)
    y = (x.float().cpu().reshape(-1, cols) * torch.from_numpy(f)).reshape(x.shape)
    return y if res is None else res.float().cpu() + y


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (2, 9), (64, 1000), (1001, 77), (7, 8192), (1, 100003)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("res", [False, True])
def test_dropout_bits(rows, cols, dtype, res):
    torch, train = _torch(), _train()
    print(f"dropout {rows}x{cols} {dtype} {res}", flush=True)
    x = torch.randn(rows, cols, device="cuda").to(_dt(dtype))
    r = torch.randn(rows, cols, device="cuda").to(_dt(dtype)) if res else None
    seed, offset = 0x123456789ABCDEF0 + rows, (5 << 32) + cols
    y = train.dropout(x, 0.3, train.Rng(seed, offset), residual=r)
    want = dropped(x, 0.3, seed, offset, r).to(_dt(dtype))
    assert torch.equal(y.cpu(), want)
    assert torch.equal(train.dropout_backward(x, 0.3, train.Rng(seed, offset)).cpu(), dropped(x, 0.3, seed, offset).to(_dt(dtype)))


def test_dropout_views_in_place_and_p_zero():
    torch, train = _torch(), _train()
    print("dropout views", flush=True)
    rng = train.Rng(3, 4)
    big = torch.randn(40, 105, device="cuda").bfloat16()
    x = big[:, 3:80]   # rows that start at odd elements
    want = dropped(x, 0.5, 3, 4).bfloat16()
    out = torch.zeros(40, 99, device="cuda").bfloat16()
    assert torch.equal(train.dropout(x, 0.5, rng, out=out[:, 1:78]).cpu(), want)
    assert (out[:, 0] == 0).all() and (out[:, 78:] == 0).all()
    y = x.contiguous()
    assert torch.equal(train.dropout(y, 0.5, rng, out=y).cpu(), want)
    assert torch.equal(train.dropout(x, 0.0, None), x)
    z = torch.randn(2, 3, 5, 8, device="cuda")
    assert torch.equal(train.dropout(z, 0.5, rng).view(30, 8), train.dropout(z.view(30, 8), 0.5, rng))
    for shape in ((0, 5), (5, 0)):
        assert train.dropout(torch.zeros(shape, device="cuda"), 0.5, rng).shape == shape
    nan = torch.full((4, 64), float("nan"), device="cuda")
    kept = torch.from_numpy(T.dropout_factor(4, 64, 0.5, 3, 4) > 0)
    assert torch.equal(train.dropout(nan, 0.5, rng).isnan().cpu(), kept)   # a dropped NaN is 0


def test_dropout_residual_in_place():
    torch, train = _torch(), _train()
    print("dropout residual in place", flush=True)
    x, r = torch.randn(50, 300, device="cuda"), torch.randn(50, 300, device="cuda")
    want = dropped(x, 0.2, 9, 1, r)
    assert torch.equal(train.dropout(x, 0.2, train.Rng(9, 1), residual=r, out=r).cpu(), want)


def test_device_offset_moves_a_replayed_graph():
    torch, train = _torch(), _train()
    print("dropout graph", flush=True)
    x = torch.randn(64, 512, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    rng = train.Rng(11, 100, step)
    train.dropout(x, 0.5, rng)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = train.dropout(x, 0.5, rng)
    for n in range(3):
        step.fill_(n)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), dropped(x, 0.5, 11, 100 + n)), n


NORM = [(1, 1), (3, 5), (9, 8), (17, 64), (130, 511), (64, 512), (33, 513), (40, 1000), (21, 1024), (10, 1032),
        (1030, 2048), (5, 2049), (7, 4096), (6, 5000), (3, 8192), (4, 8200), (2, 12289), (3, 16384), (2, 16383)]


@pytest.mark.parametrize("rows,cols", NORM)
@pytest.mark.parametrize("dtype,hd,p", [("bf16", None, 0.0), ("bf16", "bf16", 0.1), ("bf16", "f32", 0.1), ("f16", "f16", 0.0),
                                        ("f16", "f32", 0.3), ("f32", "f32", 0.0), ("f32", None, 0.2)])
def test_layer_norm(rows, cols, dtype, hd, p):
    torch, train = _torch(), _train()
    print(f"layer norm {rows}x{cols} {dtype} {hd} {p}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows * cols)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (2 * mk(rows, cols) + 0.5).to(_dt(dtype))
    res = mk(rows, cols).to(_dt(hd)) if hd else None
    w, b = 1 + 0.2 * mk(cols), mk(cols)
    rng = train.Rng(77, 5)
    eps = 1e-5
    y, h, mean, rstd = train.layer_norm_forward(x, w, b, eps=eps, residual=res, p=p, rng=rng)
    if hd is None and p == 0:
        assert h is x
    else:
        v = dropped(x, p, 77, 5, res) if p else res.float().cpu() + x.float().cpu()
        assert torch.equal(h.cpu(), v.to(h.dtype))
    H, W, B = np64(h), np64(w), np64(b)
    f = T.layer_norm(H, W, B, eps)
    scale = np.abs(H).mean(1) + 1e-30
    # var + eps may be eps alone (one column): rstd's error follows from the centred values'
    inside(np64(mean), f["mean"], 2.0 ** -19 * scale, "mean")
    inside(np64(rstd), f["rstd"], 2.0 ** -18 * f["rstd"] * (1 + f["rstd"] * scale), "rstd")
    shift = 2.0 ** -19 * (scale * f["rstd"])[:, None]   # the mean's error, in units of xh
    inside(np64(y), f["y"], U[dtype] * np.abs(f["y"]) + 2.0 ** -18 * (np.abs(f["xh"] * W) * (1 + shift * 2 ** 19 * 2 ** -1) + np.abs(B)) + shift * np.abs(W), "y")
    dy = mk(rows, cols).to(_dt(dtype))
    dh = mk(rows, cols).to(h.dtype) if hd else None
    dx, dres, dw, db = train.layer_norm_backward(dy, h, w, mean, rstd, dh=dh, p=p, rng=rng)
    DY, DH = np64(dy), np64(dh) if hd else None
    r = T.layer_norm_backward(DY, H, W, eps, DH)
    z, xh = np.abs(r["z"]), np.abs(r["xh"])
    zx = (z * xh).mean(1, keepdims=True)
    e = 2.0 ** -17 * r["rstd"][:, None] * (z + z.mean(1, keepdims=True) + (xh + 1) * zx + xh * z.mean(1, keepdims=True))
    e = e * (1 + (scale * r["rstd"])[:, None]) + (0 if DH is None else 2.0 ** -23 * np.abs(DH))
    uh = U["f32" if h.dtype == torch.float32 else dtype]
    inside(np64(dres), r["g"], uh * np.abs(r["g"]) + e, "dres")
    F = T.dropout_factor(rows, cols, p, 77, 5).astype(np.float64) if p else 1.0
    inside(np64(dx), r["g"] * F, F * ((U[dtype] + 2.0 ** -23) * np.abs(r["g"]) * 1.01 + e) + 2.0 ** -25, "dx")
    terms = (np.abs(DY) * xh).sum(0)
    shift_w = (np.abs(DY) * shift).sum(0)
    inside(np64(dw), r["dweight"], ((rows + 16) * 2.0 ** -24 + 2.0 ** -18) * terms * (1 + (scale * f["rstd"]).max()) + 2 * shift_w, "dweight")
    inside(np64(db), r["dbias"], (rows + 16) * 2.0 ** -24 * np.abs(DY).sum(0), "dbias")


def test_offset_rows_keep_their_precision():
    """Values far from zero: the variance is taken about the mean."""
    torch, train = _torch(), _train()
    print("layer norm offset", flush=True)
    x = 1000 + torch.randn(8, 2048, device="cuda")
    w = torch.ones(2048, device="cuda")
    y, _, mean, rstd = train.layer_norm_forward(x, w)
    f = T.layer_norm(np64(x), np64(w), None, 1e-5)
    # mean within a few ulp of 1000 (2^-14 each), then xh within that over sigma = 1
    assert np.max(np.abs(np64(y) - f["y"])) < 8 * 2.0 ** -14
    assert np.max(np.abs(np64(rstd) / f["rstd"] - 1)) < 1e-4


def test_views_in_place_no_bias_no_rows():
    torch, train = _torch(), _train()
    print("layer norm views", flush=True)
    w = torch.randn(77, device="cuda")
    big = torch.randn(30, 99, device="cuda").bfloat16()
    x = big[:, 5:82]
    y, h, mean, rstd = train.layer_norm_forward(x, w)
    y2, _, mean2, rstd2 = train.layer_norm_forward(x.contiguous(), w)
    assert torch.equal(y, y2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    c = x.contiguous()
    assert train.layer_norm_forward(c, w, out=c)[0] is c and torch.equal(c, y2)
    a = train.layer_norm_backward(big[:, 1:78], x, w, mean, rstd)
    b = train.layer_norm_backward(big[:, 1:78].contiguous(), x.contiguous(), w, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert a[1] is a[0] and train.layer_norm_backward(x, x, w, mean, rstd, residual_grad=False)[1] is None
    x0 = torch.zeros(0, 77, device="cuda")
    y, h, mean, rstd = train.layer_norm_forward(x0, w)
    assert y.shape == (0, 77)
    _, _, dw, db = train.layer_norm_backward(x0, h, w, mean, rstd)
    assert (dw == 0).all() and (db == 0).all()


def test_leading_axes():
    torch, train = _torch(), _train()
    print("layer norm axes", flush=True)
    x, w = torch.randn(3, 4, 64, device="cuda"), torch.randn(64, device="cuda")
    y, _, mean, rstd = train.layer_norm_forward(x, w)
    assert mean.shape == (3, 4) and torch.equal(y.view(12, 64), train.layer_norm_forward(x.view(12, 64), w)[0])
    with pytest.raises(ValueError, match="leading axes"):
        train.layer_norm_forward(x.transpose(0, 1), w)


def test_equal_bits_on_another_stream_and_in_a_graph():
    torch, train = _torch(), _train()
    print("layer norm streams", flush=True)
    x, res, w = torch.randn(3000, 1000, device="cuda").bfloat16(), torch.randn(3000, 1000, device="cuda"), torch.randn(1000, device="cuda")
    rng = train.Rng(1, 2)

    def both(stream=None):
        y, h, mean, rstd = train.layer_norm_forward(x, w, residual=res, p=0.1, rng=rng, stream=stream)
        return (y, h, mean, rstd, *train.layer_norm_backward(x, h, w, mean, rstd, dh=res, p=0.1, rng=rng, stream=stream))

    first = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = both(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = both()
    for n in range(3):
        x.copy_(torch.randn_like(x))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, both())), n


def test_more_rows_than_one_launch_holds():
    """Past 2^31 threads the rows take several launches, and the dropped bits
    go on from one to the next."""
    torch, train = _torch(), _train()
    rows, cols, part = 2 ** 27 + 3, 8, 2 ** 20
    print("norm rows", rows, flush=True)
    x = torch.randn(part, cols, device="cuda").bfloat16().repeat(rows // part + 1, 1)[:rows]
    w = torch.randn(cols, device="cuda")
    y, h, mean, rstd = train.layer_norm_forward(x, w, p=0.25, rng=train.Rng(5, 9))
    assert torch.equal(h, train.dropout(x, 0.25, train.Rng(5, 9)))
    y2, _, mean2, rstd2 = train.layer_norm_forward(h[-part:].contiguous(), w)
    assert torch.equal(y[-part:], y2) and torch.equal(mean[-part:], mean2) and torch.equal(rstd[-part:], rstd2)


def test_memory_of_a_call_on_another_stream_is_not_handed_out_early():
    """An input dropped after a call on another stream keeps its memory until that stream is past the call."""
    torch, train = _torch(), _train()
    print("dropout, dropped input", flush=True)
    x = torch.randn(3001, 5003, device="cuda")
    rng = train.Rng(3, 4)
    want = train.dropout(x, 0.3, rng)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        busy = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            busy = busy @ busy / 64
    at = x.data_ptr()
    got = train.dropout(x, 0.3, rng, stream=s)
    del x
    other = [torch.full((3001, 5003), float("nan"), device="cuda") for _ in range(3)]
    assert all(t.data_ptr() != at for t in other)
    s.synchronize()
    assert torch.equal(got, want)
