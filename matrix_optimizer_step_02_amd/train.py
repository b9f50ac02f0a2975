"""The training pass's operators on torch tensors: attention, position rotation,
norms of queries and keys, layer norm, dropout and the clipped policy loss, each
with its backward pass.

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
import math
from fractions import Fraction
from typing import NamedTuple, Optional

import torch

from . import native

__all__ = ["Rng", "attention_forward", "attention_backward", "rotary_frequencies", "Rotary", "rotary_forward",
           "rotary_backward", "qk_norm_forward", "qk_norm_backward", "dropout", "dropout_backward",
           "layer_norm_forward", "layer_norm_backward", "PolicyForward", "policy_loss_forward",
           "policy_loss_backward", "policy_loss_step"]

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


def _desc(q, k, v, causal, window, sinks, scale, q_start, k_start, max_q, max_k, q_lens, k_lens):
    if sinks >> 31:
        raise ValueError("sinks must be in [0, 2^31)")
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
                                      _vector(k_start, "k_start", dev, batch + 1, torch.int32), nq, ks[0], sinks=sinks)
        return a, dev, (heads, nq)
    batch, nq, heads, dim = qs
    a = native.opt_attention_desc(code, batch, heads, ks[2], dim, nq, ks[1], bool(causal), window,
                                  dim ** -0.5 if scale is None else scale, sinks=sinks)
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
def attention_forward(q, k, v, *, causal=False, window=0, sinks=0, scale=None, q_start=None, k_start=None, max_q=None,
                      max_k=None, q_lens=None, k_lens=None, out=None):
    """(out, lse) of softmax(scale q k^T) v. q is (batch, tokens, heads, dim);
    k and v (batch, tokens, kv_heads, dim); any strides with a contiguous last
    axis. window > 0 (with causal) hides keys that lie ``window`` or more behind
    a query, but for the sequence's first ``sinks``. Packed sequences: q, k, v without the batch axis, q_start and k_start
    int32 offsets of batch + 1, max_q and max_k the longest lengths. Padded
    batches: q_lens, k_lens int32 lengths. lse is fp32, (heads, all query
    tokens). scale defaults to dim^-1/2. Tokens outside every sequence, past a
    length or past max_q or max_k are not read; out is 0 and lse -inf there."""
    a, dev, per_row = _desc(q, k, v, causal, window, sinks, scale, q_start, k_start, max_q, max_k, q_lens, k_lens)
    st = _stream(dev)
    o = _out(out, "out", q, dev)
    lse = q.new_empty(per_row, dtype=torch.float32)
    n = native.opt_attention_workspace_size(a, 0)
    ws = _bytes(q, n)
    native.opt_attention_forward(a, _bhtd(q, "q"), _bhtd(k, "k"), _bhtd(v, "v"), _bhtd(o, "out"), lse.data_ptr(),
                                 ws.data_ptr() if n else 0, n, st)
    return o, lse


@_streamed
def attention_backward(dout, q, k, v, out, lse, *, causal=False, window=0, sinks=0, scale=None, q_start=None,
                       k_start=None, max_q=None, max_k=None, q_lens=None, k_lens=None, dq=None, dk=None, dv=None):
    """(dq, dk, dv) from the output's gradient and what attention_forward took
    and returned. dq, dk, dv may be given, for instance as views of one
    projection's gradient. They are 0 for tokens outside every sequence."""
    a, dev, per_row = _desc(q, k, v, causal, window, sinks, scale, q_start, k_start, max_q, max_k, q_lens, k_lens)
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


# --------------------------------------------------- rotary and qk norm ----


def rotary_frequencies(rot, base=10000.0, *, scaling=None, factor=1.0, original_length=0, low=1.0, high=32.0):
    """(frequencies, scale) for Rotary: f_i = base^(-2 i / rot), i < rot / 2, in
    64 bits. Scaled for contexts ``factor`` times as long:

    * "linear": f_i / factor.
    * "base": the base is raised to base factor^(rot / (rot - 2)), which divides
      the lowest frequency by factor and leaves the highest.
    * "ramp": f_i / factor for pairs that turn fewer than ``low`` times over
      ``original_length`` positions, f_i for those that turn more than ``high``
      times, linear in the number of turns between, and scale = 1 + 0.1 ln factor
      (Peng, Quesnel, Fan, Shippole: "YaRN", 2023)."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and >= 2")
    if not (base > 0 and math.isfinite(base)):
        raise ValueError("base must be positive and finite")
    if scaling is not None and not (factor >= 1 and math.isfinite(factor)):
        raise ValueError("factor must be >= 1 and finite")
    if scaling == "base":
        if rot == 2:
            raise ValueError("scaling of the base needs rot > 2")
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling in (None, "base"):
        return f, 1.0
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling != "ramp":
        raise ValueError(f"scaling is {scaling!r}, expected None, 'linear', 'base' or 'ramp'")
    if not (original_length > 0 and high > low):
        raise ValueError("scaling by a ramp needs original_length > 0 and high > low")
    keep = [min(max((x * original_length / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for x in f]
    return [x * k + x / factor * (1 - k) for x, k in zip(f, keep)], 1.0 + 0.1 * math.log(factor)


_TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
_TURN = round((1 << 256) / _TWO_PI)


def _turns(f: float) -> int:
    """2^64 f / (2 pi), rounded and reduced to one turn: f is n / 2^k."""
    n, d = f.as_integer_ratio()
    shift = 256 - 64 + d.bit_length() - 1
    return ((n * _TURN + (1 << (shift - 1))) >> shift) % (1 << 64)


_WIDE = {torch.int32: 0, torch.int64: 1}


class _Rotary(NamedTuple):
    turns: torch.Tensor
    rot: int
    layout: int
    scale: float
    device: torch.device
    ptr: int


class Rotary(_Rotary):
    """What turns queries and keys: a program makes it once. ``frequencies``:
    radians a position, one per pair (2 len(frequencies) elements of a head are
    turned). layout "half" pairs element i with i + rot / 2, "pairs" 2 i with
    2 i + 1. ``scale``: factor of cosine and sine."""

    def __new__(cls, frequencies, *, layout="half", scale=1.0, device="cuda"):
        if layout not in ("half", "pairs"):
            raise ValueError(f"layout is {layout!r}, expected 'half' or 'pairs'")
        f = [float(x) for x in frequencies]
        if not f or not all(math.isfinite(x) for x in f):
            raise ValueError("frequencies must be finite, one at least")
        if not (scale > 0 and math.isfinite(scale)):
            raise ValueError("scale must be positive and finite")
        turns = [_turns(x) for x in f]   # as the two's complement that int64 holds
        table = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device)
        code = native.OPT_ROTARY_HALF if layout == "half" else native.OPT_ROTARY_PAIRS
        return cls._of(table, code, float(scale))

    @classmethod
    def _of(cls, table, code, scale):
        return super().__new__(cls, table, 2 * table.numel(), code, scale, table.device, table.data_ptr())

    def __reduce__(self):   # copies and pickles: a table of their own has another address
        return Rotary._of, (self.turns, self.layout, self.scale)

    def c(self, positions, first, qs, dev):
        """The descriptor for the tokens of queries of shape qs."""
        turns, rot, layout, scale, device, ptr = self
        if device != dev:
            raise ValueError(f"rope is on {device}, expected {dev}")
        if positions is None:
            return native.opt_rotary(ptr, rot, layout, scale, 0, 0, 0, 0, first)
        if first:
            raise ValueError("first goes without positions")
        if not isinstance(positions, torch.Tensor):
            raise ValueError("positions must be an int32 or int64 tensor")
        wide = _WIDE.get(positions.dtype)
        if wide is None:
            raise ValueError("positions must be an int32 or int64 tensor")
        shape, s, b = positions.shape, positions.stride(), 0
        if len(shape) == 2:
            ok, b = len(qs) == 4 and shape[0] == qs[0] and shape[1] == qs[1], s[0]
        else:
            ok = len(shape) == 1 and shape[0] == qs[-3]
        if not ok or positions.device != dev:
            _is(positions, "positions", dev, positions.dtype, qs[:-2])
        return native.opt_rotary(ptr, rot, layout, scale, wide, positions.data_ptr(), b, s[-1])


def _heads(q, k, q_name, k_name):
    """The descriptor of queries and keys (k may be None), q's shape and device."""
    qs, dev, kv = q.shape, q.device, 0
    if len(qs) == 4:
        batch, tokens, heads, dim = qs
    elif len(qs) == 3:
        batch, (tokens, heads, dim) = 1, qs
    else:
        raise ValueError(f"{q_name} must have axes (batch, tokens, heads, dim) or (tokens, heads, dim)")
    code = _code(q, q_name)
    if k is not None:
        ks = k.shape
        if not (k.dtype is q.dtype and k.device == dev and len(ks) == len(qs) and ks[-1] == dim
                and ks[-3] == tokens and ks[0] == qs[0]):
            _is(k, k_name, dev, q.dtype)
            raise ValueError(f"{k_name} has shape {tuple(ks)}, expected {tuple(qs)} but for the heads")
        kv = ks[-2]
    return native.opt_heads_desc(code, heads, kv, dim, batch, tokens), qs, dev


def _like(t, name, like):
    """The given result, or a new one."""
    if t is None:
        return torch.empty_like(like)
    if not (t.dtype is like.dtype and t.device == like.device and t.shape == like.shape):
        _is(t, name, like.device, like.dtype, like.shape)
    return t


def _rotary(names, q, k, rope, positions, first, out_q, out_k, inverse):
    d, qs, dev = _heads(q, k, names[0], names[1])
    if inverse:   # a gradient may have any strides: 0 where it is expanded, others behind a transposition
        if q.stride(-1) != 1:
            q = q.contiguous()
        if k is not None and k.stride(-1) != 1:
            k = k.contiguous()
    if rope.__class__ is not Rotary:
        raise TypeError("rope must be a Rotary")
    r = rope.c(positions, first, qs, dev)
    st = _stream(dev)
    yq = _like(out_q, names[2], q)
    if k is None:
        native.opt_rotary_apply(d, r, inverse, _bhtd(q, names[0]), None, _bhtd(yq, names[2]), None, st)
        return yq, None
    yk = _like(out_k, names[3], k)
    native.opt_rotary_apply(d, r, inverse, _bhtd(q, names[0]), _bhtd(k, names[1]), _bhtd(yq, names[2]),
                            _bhtd(yk, names[3]), st)
    return yq, yk


@_streamed
def rotary_forward(q, k, rope, positions=None, *, first=0, out_q=None, out_k=None):
    """(yq, yk): queries (batch, tokens, heads, dim) and keys (batch, tokens,
    kv_heads, dim), or both without the batch axis, turned by ``rope`` at their
    positions: an int32 or int64 tensor (batch, tokens) or (tokens,), or first + the
    index along the tokens. k may be None. out_q may be q and out_k may be k."""
    return _rotary(("q", "k", "out_q", "out_k"), q, k, rope, positions, first, out_q, out_k, 0)


@_streamed
def rotary_backward(dyq, dyk, rope, positions=None, *, first=0, dq=None, dk=None):
    """(dq, dk) from the gradients of rotary_forward's results. dq and dk may be
    given, for instance as views of one projection's gradient, or be dyq and dyk."""
    return _rotary(("dyq", "dyk", "dq", "dk"), dyq, dyk, rope, positions, first, dq, dk, 1)


def _rope(rope, positions, first, qs, dev):
    if rope is None:
        if positions is not None or first:
            raise ValueError("positions go with a rope")
        return None
    if rope.__class__ is not Rotary:
        raise TypeError("rope must be a Rotary or None")
    return rope.c(positions, first, qs, dev)


@_streamed
def qk_norm_forward(q, k, q_weight, k_weight, *, eps=1e-6, rope=None, positions=None, first=0, out_q=None, out_k=None):
    """(yq, yk, q_rstd, k_rstd): each head's row divided by its root mean square
    and multiplied by a weight (dim, fp32; one for queries, one for keys), then
    turned as rotary_forward turns it (rope None: not turned). k may be None, and
    with it what belongs to keys. out_q may be q and out_k may be k (but the
    backward pass needs q and k)."""
    d, qs, dev = _heads(q, k, "q", "k")
    r = _rope(rope, positions, first, qs, dev)
    dim = qs[-1]
    wq = _vector(q_weight, "q_weight", dev, dim)
    wk = 0 if k is None else _vector(k_weight, "k_weight", dev, dim)
    st = _stream(dev)
    yq = _like(out_q, "out_q", q)
    q_rstd = q_weight.new_empty(qs[:-1])
    if k is None:
        native.opt_qk_norm_forward(d, r, _bhtd(q, "q"), None, wq, 0, eps, _bhtd(yq, "out_q"), None,
                                   q_rstd.data_ptr(), 0, st)
        return yq, None, q_rstd, None
    yk = _like(out_k, "out_k", k)
    k_rstd = q_weight.new_empty(k.shape[:-1])
    native.opt_qk_norm_forward(d, r, _bhtd(q, "q"), _bhtd(k, "k"), wq, wk, eps, _bhtd(yq, "out_q"), _bhtd(yk, "out_k"),
                               q_rstd.data_ptr(), k_rstd.data_ptr(), st)
    return yq, yk, q_rstd, k_rstd


def _statistic(t, name, dev, shape):
    if not (t.dtype == torch.float32 and t.device == dev and t.shape == shape):
        _is(t, name, dev, torch.float32, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


@_streamed
def qk_norm_backward(dyq, dyk, q, k, q_weight, k_weight, q_rstd, k_rstd, *, rope=None, positions=None, first=0, dq=None,
                     dk=None):
    """(dq, dk, dq_weight, dk_weight) from the gradients of qk_norm_forward's
    results, what it took and the rstd it returned. dq and dk may be given, for
    instance as views of one projection's gradient, or be dyq and dyk."""
    d, qs, dev = _heads(q, k, "q", "k")
    r = _rope(rope, positions, first, qs, dev)
    if dyq is None or (dyk is None) != (k is None):
        raise ValueError("dyq goes with q and dyk with k")
    dyq = _like(dyq, "dyq", q)
    dyk = dyk if k is None else _like(dyk, "dyk", k)
    if dyq.stride(-1) != 1:   # an expanded gradient has stride 0
        dyq = dyq.contiguous()
    if k is not None and dyk.stride(-1) != 1:
        dyk = dyk.contiguous()
    dim = qs[-1]
    wq, wk = _vector(q_weight, "q_weight", dev, dim), 0 if k is None else _vector(k_weight, "k_weight", dev, dim)
    sq = _statistic(q_rstd, "q_rstd", dev, qs[:-1])
    sk = 0 if k is None else _statistic(k_rstd, "k_rstd", dev, k.shape[:-1])
    st = _stream(dev)
    gq = _like(dq, "dq", q)
    gwq = torch.empty_like(q_weight)
    n = native.opt_qk_norm_workspace_size(d)
    ws = _bytes(q, n)
    wp = ws.data_ptr() if n else 0
    if k is None:
        native.opt_qk_norm_backward(d, r, _bhtd(dyq, "dyq"), None, _bhtd(q, "q"), None, wq, 0, sq, 0, _bhtd(gq, "dq"),
                                    None, gwq.data_ptr(), 0, wp, n, st)
        return gq, None, gwq, None
    gk = _like(dk, "dk", k)
    gwk = torch.empty_like(k_weight)
    native.opt_qk_norm_backward(d, r, _bhtd(dyq, "dyq"), _bhtd(dyk, "dyk"), _bhtd(q, "q"), _bhtd(k, "k"), wq, wk, sq, sk,
                                _bhtd(gq, "dq"), _bhtd(gk, "dk"), gwq.data_ptr(), gwk.data_ptr(), wp, n, st)
    return gq, gk, gwq, gwk


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
