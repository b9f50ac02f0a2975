"""The training pass's operators on torch tensors: attention, layer norm,
dropout and the clipped policy loss, each with its backward pass.

Functions check their tensors, allocate what they return and call the C entry
points of include/matopt_train.h on the current stream, or on the one given as
``stream``. There is no autograd graph: a backward function is called with what its
forward function returned, and its results are ordinary tensors (a weight's
gradient goes into the G of a RotatedAdamGroup). Tensors that require a
gradient are therefore refused, except under torch.no_grad(). All shapes and
argument errors raise before anything is launched.
"""

from __future__ import annotations

import functools
from typing import NamedTuple, Optional

import torch

from . import native

__all__ = ["Rng", "attention_forward", "attention_backward", "dropout", "dropout_backward", "layer_norm_forward",
           "layer_norm_backward", "PolicyForward", "policy_loss_forward", "policy_loss_backward", "policy_loss_step"]

_HALF = {torch.bfloat16: native.OPT_BF16, torch.float16: native.OPT_F16}
_DTYPE = {torch.float32: native.OPT_F32, torch.bfloat16: native.OPT_BF16, torch.float16: native.OPT_F16}


class Rng(NamedTuple):
    """Where dropout's random bits come from: the same (seed, offset) give the
    same mask. ``device_offset``: an int64 tensor of one element added to
    offset on the device, for a step counter that a replayed graph reads."""
    seed: int
    offset: int = 0
    device_offset: Optional[torch.Tensor] = None

    def c(self) -> native.opt_rng:
        d = self.device_offset
        if d is not None and (d.dtype != torch.int64 or d.numel() != 1 or d.device.type != "cuda"):
            raise ValueError("device_offset must be one int64 element on a HIP device")
        m = (1 << 64) - 1
        return native.opt_rng(self.seed & m, self.offset & m, d.data_ptr() if d is not None else 0)


def _tensors(values):
    for x in values:
        if isinstance(x, torch.Tensor):
            yield x
        elif isinstance(x, tuple):   # Rng, PolicyForward
            yield from _tensors(x)
            yield from _tensors((getattr(x, "lse_rest", None),))


def _streamed(fn):
    """Gives fn a ``stream`` argument. Everything of the call happens there:
    the kernels, the copies it may need, and the allocation of what it returns
    (so that no memory is taken that the current stream may still be using).
    The tensors it was given are recorded on that stream: their memory is not
    handed out again before the stream is past the call. It does not wait for
    what writes them, nor the current stream for its results."""
    needs_no_grad = (f"{fn.__name__} keeps no graph for a tensor that requires a gradient: call it under "
                     "torch.no_grad(), and the backward function for the gradient")
    grad_enabled, tensor = torch.is_grad_enabled, torch.Tensor

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if grad_enabled():
            for t in args:
                if isinstance(t, tensor) and t.requires_grad:
                    raise ValueError(needs_no_grad)
            for t in kw.values():
                if isinstance(t, tensor) and t.requires_grad:
                    raise ValueError(needs_no_grad)
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            result = fn(*args, **kw)
        for t in _tensors((*args, *kw.values())):
            if t.is_cuda:
                t.record_stream(stream)
        return result
    return call


def _stream(dev):
    """The raw handle of the current stream: the Stream object around it costs
    2 us a call. The kernels go to the current device."""
    if dev.type != "cuda":
        raise ValueError("tensors must live on a HIP device")
    if dev.index != torch._C._cuda_getDevice():
        raise ValueError(f"tensors are on {dev}, which is not the current device (torch.cuda.device)")
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _is(t, name, device, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _vector(t, name, device, n, dtype=torch.float32):
    if not (t.__class__ is torch.Tensor and t.dtype == dtype and t.device == device and t.shape == (n,)):
        _is(t, name, device, dtype, (n,))
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _code(t, name):
    try:
        return _DTYPE[t.dtype]
    except KeyError:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {tuple(_DTYPE)}") from None


# -------------------------------------------------------------- attention ----


def _refuse_qkv(q, k, v, packed):
    """Why q, k, v do not go together."""
    dev, dt = q.device, q.dtype
    want = 3 if packed else 4
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _is(t, name, dev, dt)
        if t.dim() != want:
            raise ValueError(f"{name} must have {want} axes: " + ("(tokens, heads, dim)" if packed else
                                                                  "(batch, tokens, heads, dim)"))
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    if q.shape[-1] != k.shape[-1]:
        raise ValueError("q and k differ in head_dim")
    if not packed and k.shape[0] != q.shape[0]:
        raise ValueError("q and k differ in batch")
    raise ValueError(f"q has dtype {dt}, expected torch.bfloat16 or torch.float16")


def _desc(q, k, v, causal, window, scale, q_start, k_start, max_q, max_k, q_lens, k_lens):
    packed = q_start is not None
    if packed != (k_start is not None):
        raise ValueError("q_start and k_start come together")
    dev, dt, qs, ks = q.device, q.dtype, q.shape, k.shape
    code = _HALF.get(dt)
    if not (code is not None and k.dtype == dt == v.dtype and k.device == dev == v.device and ks == v.shape
            and len(qs) == len(ks) == (3 if packed else 4) and qs[-1] == ks[-1] and (packed or qs[0] == ks[0])):
        _refuse_qkv(q, k, v, packed)
    if packed:
        if q_lens is not None or k_lens is not None:
            raise ValueError("packed sequences (q_start) have no q_lens or k_lens")
        if max_q is None or max_k is None:
            raise ValueError("packed sequences need max_q and max_k")
        nq, heads, dim = qs
        batch = q_start.numel() - 1
        a = native.opt_attention_desc(code, batch, heads, ks[1], dim, max_q, max_k, bool(causal), window,
                                      dim ** -0.5 if scale is None else scale,
                                      _vector(q_start, "q_start", dev, batch + 1, torch.int32),
                                      _vector(k_start, "k_start", dev, batch + 1, torch.int32), nq, ks[0])
        return a, dev, (heads, nq)
    batch, nq, heads, dim = qs
    a = native.opt_attention_desc(code, batch, heads, ks[2], dim, nq, ks[1], bool(causal), window,
                                  dim ** -0.5 if scale is None else scale)
    if q_lens is not None:
        a.q_lens = _vector(q_lens, "q_lens", dev, batch, torch.int32)
    if k_lens is not None:
        a.k_lens = _vector(k_lens, "k_lens", dev, batch, torch.int32)
    return a, dev, (heads, batch * nq)


def _bhtd(t, name):
    s = t.stride()
    if s[-1] != 1 and t.shape[-1] != 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    if len(s) == 3:
        return native.opt_attention_tensor(t.data_ptr(), 0, s[0], s[1])
    return native.opt_attention_tensor(t.data_ptr(), s[0], s[1], s[2])


def _out(given, name, like, dev):
    if given is None:
        return like.new_empty(like.shape)
    _is(given, name, dev, like.dtype, like.shape)
    return given


def _bytes(like, n):
    return like.new_empty(n, dtype=torch.uint8) if n else None


@_streamed
def attention_forward(q, k, v, *, causal=False, window=0, scale=None, q_start=None, k_start=None, max_q=None,
                      max_k=None, q_lens=None, k_lens=None, out=None):
    """(out, lse) of softmax(scale q k^T) v. q is (batch, tokens, heads, dim);
    k and v (batch, tokens, kv_heads, dim); any strides with a contiguous last
    axis. Packed sequences: q, k, v without the batch axis, q_start and k_start
    int32 offsets of batch + 1, max_q and max_k the longest lengths. Padded
    batches: q_lens, k_lens int32 lengths. lse is fp32, (heads, all query
    tokens). scale defaults to dim^-1/2. Tokens outside every sequence, past a
    length or past max_q or max_k are not read; out is 0 and lse -inf there."""
    a, dev, per_row = _desc(q, k, v, causal, window, scale, q_start, k_start, max_q, max_k, q_lens, k_lens)
    st = _stream(dev)
    o = _out(out, "out", q, dev)
    lse = q.new_empty(per_row, dtype=torch.float32)
    n = native.opt_attention_workspace_size(a, 0)
    ws = _bytes(q, n)
    native.opt_attention_forward(a, _bhtd(q, "q"), _bhtd(k, "k"), _bhtd(v, "v"), _bhtd(o, "out"), lse.data_ptr(),
                                 ws.data_ptr() if n else 0, n, st)
    return o, lse


@_streamed
def attention_backward(dout, q, k, v, out, lse, *, causal=False, window=0, scale=None, q_start=None, k_start=None,
                       max_q=None, max_k=None, q_lens=None, k_lens=None, dq=None, dk=None, dv=None):
    """(dq, dk, dv) from the output's gradient and what attention_forward took
    and returned. dq, dk, dv may be given, for instance as views of one
    projection's gradient. They are 0 for tokens outside every sequence."""
    a, dev, per_row = _desc(q, k, v, causal, window, scale, q_start, k_start, max_q, max_k, q_lens, k_lens)
    for t, name in ((dout, "dout"), (out, "out")):
        if not (t.dtype == q.dtype and t.device == dev and t.shape == q.shape):
            _is(t, name, dev, q.dtype, q.shape)
    _is(lse, "lse", dev, torch.float32, per_row)
    if not lse.is_contiguous():
        raise ValueError("lse must be contiguous")
    if dout.stride(-1) != 1:   # an expanded gradient has stride 0
        dout = dout.contiguous()
    st = _stream(dev)
    gq, gk, gv = _out(dq, "dq", q, dev), _out(dk, "dk", k, dev), _out(dv, "dv", v, dev)
    n = native.opt_attention_workspace_size(a, 1)
    ws = _bytes(q, n)
    native.opt_attention_backward(a, _bhtd(dout, "dout"), _bhtd(q, "q"), _bhtd(k, "k"), _bhtd(v, "v"),
                                  _bhtd(out, "out"), lse.data_ptr(), _bhtd(gq, "dq"), _bhtd(gk, "dk"),
                                  _bhtd(gv, "dv"), ws.data_ptr() if n else 0, n, st)
    return gq, gk, gv


# ---------------------------------------------------------------- dropout ----


def _rows(t, name):
    """(data pointer, row stride) of a tensor as rows x cols over its last
    axis; the leading axes must collapse to one stride."""
    shape = t.shape
    if t.is_contiguous():
        return t.data_ptr(), shape[-1] if shape else 1
    if len(shape) == 2:
        s0, s1 = t.stride()
        if s1 != 1 and shape[1] > 1:
            raise ValueError(f"the last axis of {name} must be contiguous")
        return t.data_ptr(), s0 if shape[0] > 1 else max(s0, shape[1])
    if len(shape) < 2:
        raise ValueError(f"{name} must be contiguous")
    try:
        v = t.view(-1, shape[-1])
    except RuntimeError:
        raise ValueError(f"the leading axes of {name} must collapse to one stride") from None
    return _rows(v, name)


def _size(t):
    shape = t.shape
    if len(shape) == 2:
        return shape[0], shape[1]
    cols = shape[-1] if shape else 1
    return (t.numel() // cols if cols else 0), cols


def _p_rng(p, rng, dev):
    if p > 0 and rng is None:
        raise ValueError("dropout needs an rng")
    if rng is None or not p > 0:
        return None
    c = rng.c()
    if rng.device_offset is not None and rng.device_offset.device != dev:
        raise ValueError(f"device_offset is on {rng.device_offset.device}, expected {dev}")
    return c


@_streamed
def dropout(x, p, rng, *, residual=None, out=None):
    """residual + dropout(x) (no residual: dropout(x)); out may be x or
    residual. The mask depends on rng and on an element's position in x
    (leading axes as rows, the last axis as columns)."""
    dev, dt, bits = x.device, _code(x, "x"), _p_rng(p, rng, x.device)
    rows, cols = _size(x)
    y = _out(out, "out", x, dev)
    xp, ldx = _rows(x, "x")
    yp, ldy = _rows(y, "out")
    rp, ldr = 0, 0
    if residual is not None:
        _is(residual, "residual", dev, x.dtype, x.shape)
        rp, ldr = _rows(residual, "residual")
    st = _stream(dev)
    native.opt_dropout(rows, cols, dt, xp, ldx, rp, ldr, yp, ldy, p, bits, st)
    return y


@_streamed
def dropout_backward(dy, p, rng, *, out=None):
    """dropout's gradient with respect to x (the residual's is dy itself)."""
    return dropout(dy, p, rng, out=out)


# ------------------------------------------------------------- layer norm ----


@_streamed
def layer_norm_forward(x, weight, bias=None, *, eps=1e-5, residual=None, p=0.0, rng=None, out=None):
    """(y, h, mean, rstd): h = residual + dropout(x) in the residual's type,
    y its norm over the last axis in x's type. Without residual and dropout h
    is x. weight and bias are fp32."""
    dev, dt, bits = x.device, _code(x, "x"), _p_rng(p, rng, x.device)
    rows, cols = _size(x)
    y = _out(out, "out", x, dev)
    xp, ldx = _rows(x, "x")
    yp, ldy = _rows(y, "out")
    wp = _vector(weight, "weight", dev, cols)
    bp = _vector(bias, "bias", dev, cols) if bias is not None else 0
    h, hp, ldh, rp, ldr, hdt = x, 0, 0, 0, 0, dt
    if residual is not None or p > 0:
        if residual is not None:
            hdt = _code(residual, "residual")
            _is(residual, "residual", dev, residual.dtype, x.shape)
            rp, ldr = _rows(residual, "residual")
        h = (x if residual is None else residual).new_empty(x.shape)
        hp, ldh = h.data_ptr(), cols
    lead = x.shape[:-1]
    mean, rstd = weight.new_empty(lead), weight.new_empty(lead)
    st = _stream(dev)
    native.opt_layer_norm_forward(rows, cols, dt, xp, ldx, hdt, rp, ldr, wp, bp, eps, p, bits, yp, ldy, hp, ldh,
                                  mean.data_ptr(), rstd.data_ptr(), st)
    return y, h, mean, rstd


@_streamed
def layer_norm_backward(dy, h, weight, mean, rstd, *, dh=None, p=0.0, rng=None, residual_grad=True):
    """(dx, dres, dweight, dbias) from y's gradient and what
    layer_norm_forward returned; dh is the gradient that reaches h past the
    norm. dres, h's gradient, goes to the residual; without dropout and in the
    same type it is dx itself. residual_grad=False: dres is None."""
    dev, dt, bits = dy.device, _code(dy, "dy"), _p_rng(p, rng, dy.device)
    rows, cols = _size(dy)
    hdt, shape = _code(h, "h"), dy.shape
    if not (h.device == dev and h.shape == shape):
        _is(h, "h", dev, h.dtype, shape)
    dyp, lddy = _rows(dy, "dy")
    hp, ldh = _rows(h, "h")
    wp = _vector(weight, "weight", dev, cols)
    lead = shape[:-1]
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if not (t.dtype == torch.float32 and t.device == dev and t.shape == lead):
            _is(t, name, dev, torch.float32, lead)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    dhp, lddh = 0, 0
    if dh is not None:
        _is(dh, "dh", dev, h.dtype, shape)
        dhp, lddh = _rows(dh, "dh")
    dx = dy.new_empty(shape)
    dres, drp, lddr = None, 0, 0
    if residual_grad:
        if p == 0 and h.dtype == dy.dtype:
            dres = dx
        else:
            dres = h.new_empty(shape)
            drp, lddr = dres.data_ptr(), cols
    n = native.opt_layer_norm_workspace_size(rows, cols)
    ws = _bytes(dy, n)
    dw, db = weight.new_empty(cols), weight.new_empty(cols)
    st = _stream(dev)
    native.opt_layer_norm_backward(rows, cols, dt, dyp, lddy, hdt, hp, ldh, dhp, lddh, wp, mean.data_ptr(),
                                   rstd.data_ptr(), p, bits, dx.data_ptr(), cols, drp, lddr, dw.data_ptr(),
                                   db.data_ptr(), ws.data_ptr() if n else 0, n, st)
    return dx, dres, dw, db


# ------------------------------------------------------------ policy loss ----


class _PolicyForward(NamedTuple):
    loss: torch.Tensor
    logp: torch.Tensor
    lse: torch.Tensor
    slope: torch.Tensor


class PolicyForward(_PolicyForward):
    """What policy_loss_forward returns: the loss (a scalar tensor) and per
    row the target's log probability, the log-sum and d loss / d logp. Beside
    these four it holds what policy_loss_backward takes from the same call:
    ``lse_rest``, what lse's rounding left out, and ``logit_scale`` (None:
    nothing is known of them)."""
    lse_rest: Optional[torch.Tensor] = None
    logit_scale: Optional[float] = None

    def _replace(self, **kw):
        new = super()._replace(**kw)
        new.__dict__.update(self.__dict__)
        return new


def _policy(logits, target, clip_low, clip_high, kl_coef, logit_scale):
    if logits.dim() != 2:
        raise ValueError("logits must have 2 axes (rows, vocab)")
    dev = logits.device
    rows, vocab = logits.shape
    ptr, ld = _rows(logits, "logits")
    if not isinstance(target, torch.Tensor) or target.dtype not in (torch.int32, torch.int64):
        raise ValueError("target must be an int32 or int64 tensor")
    tp = _vector(target, "target", dev, rows, target.dtype)
    a = native.opt_policy_desc(_code(logits, "logits"), target.dtype == torch.int64, rows, vocab, ld, logit_scale,
                               clip_low, clip_high, kl_coef)
    return a, dev, ptr, tp


def _policy_rows(tp, dev, n, old_logp, ref_logp, advantage, weight, kl_coef):
    if ref_logp is None and kl_coef != 0:
        raise ValueError("kl_coef needs ref_logp")
    return native.opt_policy_rows(tp, _vector(old_logp, "old_logp", dev, n),
                                  _vector(ref_logp, "ref_logp", dev, n) if ref_logp is not None else 0,
                                  _vector(advantage, "advantage", dev, n), _vector(weight, "weight", dev, n))


@_streamed
def policy_loss_forward(logits, target, old_logp, advantage, weight, *, ref_logp=None, clip_low=0.2, clip_high=0.2,
                        kl_coef=0.0, logit_scale=1.0):
    """PolicyForward of the clipped policy loss with a KL term to a reference
    policy: per row of logits (rows, vocab) a target token, its log
    probability under the sampling and the reference policy, an advantage and
    a weight (which holds the normalisation; 0 leaves the row out)."""
    a, dev, lp, tp = _policy(logits, target, clip_low, clip_high, kl_coef, logit_scale)
    rows = _policy_rows(tp, dev, a.rows, old_logp, ref_logp, advantage, weight, kl_coef)
    st = _stream(dev)
    n = native.opt_policy_loss_workspace_size(a)
    ws = _bytes(logits, n)
    loss, logp, lse, slope, rest = (weight.new_empty(s) for s in ((), a.rows, a.rows, a.rows, a.rows))
    a.lse_rest = rest.data_ptr()
    native.opt_policy_loss_forward(a, lp, rows, loss.data_ptr(), logp.data_ptr(), lse.data_ptr(), slope.data_ptr(),
                                   ws.data_ptr() if n else 0, n, st)
    f = PolicyForward(loss, logp, lse, slope)
    f.lse_rest, f.logit_scale = rest, logit_scale
    return f


@_streamed
def policy_loss_backward(logits, target, fwd, *, grad=None, logit_scale=None, out=None):
    """dlogits from policy_loss_forward's result; grad: the loss's gradient, a
    scalar tensor on the device (None: 1). logit_scale is the forward call's
    and may be left out. out may be logits."""
    scale = getattr(fwd, "logit_scale", None)
    if logit_scale is None:
        logit_scale = 1.0 if scale is None else scale
    elif scale is not None and logit_scale != scale:
        raise ValueError(f"logit_scale is {logit_scale}, the forward call's was {scale}")
    a, dev, lp, tp = _policy(logits, target, 0.2, 0.2, 0.0, logit_scale)
    d = _out(out, "out", logits, dev)
    dp, ldd = _rows(d, "out")
    sp, ep = _vector(fwd.slope, "slope", dev, a.rows), _vector(fwd.lse, "lse", dev, a.rows)
    rest = getattr(fwd, "lse_rest", None)
    if rest is not None:
        a.lse_rest = _vector(rest, "lse_rest", dev, a.rows)
    gp = 0
    if grad is not None:
        _is(grad, "grad", dev, torch.float32, ())
        gp = grad.data_ptr()
    st = _stream(dev)
    native.opt_policy_loss_backward(a, lp, tp, ep, sp, gp, dp, ldd, st)
    return d


@_streamed
def policy_loss_step(logits, target, old_logp, advantage, weight, *, ref_logp=None, clip_low=0.2, clip_high=0.2,
                     kl_coef=0.0, logit_scale=1.0, grad=1.0, out=None):
    """(loss, logp, dlogits) in one pass over the logits, for a loss that is
    the last operator: grad, the loss's own gradient, is a number. out may be
    logits."""
    a, dev, lp, tp = _policy(logits, target, clip_low, clip_high, kl_coef, logit_scale)
    rows = _policy_rows(tp, dev, a.rows, old_logp, ref_logp, advantage, weight, kl_coef)
    d = _out(out, "out", logits, dev)
    dp, ldd = _rows(d, "out")
    st = _stream(dev)
    logp, loss = weight.new_empty(a.rows), weight.new_empty(())
    n = native.opt_policy_loss_workspace_size(a)
    ws = _bytes(logits, n)
    native.opt_policy_loss_step(a, lp, rows, grad, loss.data_ptr(), logp.data_ptr(), dp, ldd,
                                ws.data_ptr() if n else 0, n, st)
    return loss, logp, d
