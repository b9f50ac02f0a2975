"""The AdamW step over many tensors at once (include/matopt_adamw.h): for the
parameters that are no matrix for RotatedAdamGroup, such as embeddings, norm
weights and biases."""

from __future__ import annotations

from dataclasses import dataclass
from typing import NamedTuple, Optional, Sequence

import torch

from . import native
from .train import Rng

__all__ = ["AdamWGroup", "AdamWHyper", "GradNorm", "adamw_state"]

_DTYPE = {torch.float32: native.OPT_F32, torch.bfloat16: native.OPT_BF16, torch.float16: native.OPT_F16}
_M8, _V8 = torch.float8_e4m3fn, torch.float8_e5m2


@dataclass
class AdamWHyper:
    lr: float = 1e-3
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.0   # of the tensors that do not name their own

    def c(self) -> native.opt_adamw_hparams:
        return native.opt_adamw_hparams(self.lr, self.beta1, self.beta2, self.eps)


class GradNorm(NamedTuple):
    """The gradients' 2-norm, and the factor that clips it (NaN where it is not finite): scalars on the device."""
    norm: torch.Tensor
    scale: torch.Tensor


def _blocks(n: int) -> int:
    return -(-n // native.OPT_ADAMW_BLOCK)


def adamw_state(W: torch.Tensor, bits: int = 32) -> dict:
    """Fresh moments of one tensor: m and v in fp32, or in 8 bits with a scale per 256
    elements (which move less than in fp32 where their gradients stay 2^15 below the
    largest of the 256)."""
    if bits == 32:
        return {"m": torch.zeros_like(W, dtype=torch.float32), "v": torch.zeros_like(W, dtype=torch.float32)}
    if bits != 8:
        raise ValueError("bits must be 32 or 8")
    zeros = lambda dt: torch.zeros(W.shape, dtype=torch.uint8, device=W.device).view(dt)  # noqa: E731
    scale = lambda: torch.zeros(_blocks(W.numel()), device=W.device)  # noqa: E731
    return {"m": zeros(_M8), "v": zeros(_V8), "m_scale": scale(), "v_scale": scale()}


def _check(t, name, shape, dtypes, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_KEYS = {"W", "G", "m", "v", "m_scale", "v_scale", "W16", "lr_scale", "weight_decay"}


def make_adamw_desc(p: dict, hp: AdamWHyper) -> native.opt_adamw_desc:
    """Descriptor of one tensor from a dict as AdamWGroup takes them."""
    if p.keys() - _KEYS:
        raise ValueError(f"unknown keys {sorted(p.keys() - _KEYS)}")
    W, G, m, v = p["W"], p["G"], p["m"], p["v"]
    if not isinstance(W, torch.Tensor):
        raise TypeError("W must be a torch.Tensor")
    dev, shape, n = W.device, W.shape, W.numel()
    _check(W, "W", shape, (torch.float32,), dev)
    _check(G, "G", shape, _DTYPE, dev)
    narrow = isinstance(m, torch.Tensor) and m.dtype != torch.float32
    _check(m, "m", shape, (_M8,) if narrow else (torch.float32,), dev)
    _check(v, "v", shape, (_V8,) if narrow else (torch.float32,), dev)
    for key in ("m_scale", "v_scale"):
        if narrow:
            _check(p.get(key), key, (_blocks(n),), (torch.float32,), dev)
        elif p.get(key) is not None:
            raise ValueError(f"{key} goes with states of 8 bits")
    w16 = p.get("W16")
    if w16 is not None:
        _check(w16, "W16", shape, (torch.bfloat16, torch.float16), dev)
    ptr = lambda t: t.data_ptr() if t is not None else 0  # noqa: E731
    decay = p.get("weight_decay")
    return native.opt_adamw_desc(n, W.data_ptr(), G.data_ptr(), _DTYPE[G.dtype], 8 if narrow else 32, m.data_ptr(),
                                 v.data_ptr(), ptr(p.get("m_scale")), ptr(p.get("v_scale")), ptr(w16),
                                 _DTYPE[w16.dtype] if w16 is not None else 0, p.get("lr_scale", 1.0),
                                 hp.weight_decay if decay is None else decay)


class AdamWGroup:
    """Tensors stepped together by AdamW in one launch per kind of state.

    ``params``: a sequence of dicts with W (fp32), G (fp32, bf16 or fp16; the caller
    writes each step's gradient into it), m and v (adamw_state: fp32, or
    float8_e4m3fn and float8_e5m2 with m_scale and v_scale), and, where wanted, W16 (a bf16
    or fp16 copy of W that each step writes), weight_decay and lr_scale. All
    tensors are the caller's, contiguous, on the current device, and referenced here.
    The order of the tensors is part of what 8-bit states are rounded by.

    A group outlives the graphs that its calls are captured into. Its calls share a
    workspace: two of them on different streams are the caller's to order."""

    def __init__(self, params: Sequence[dict], hp: Optional[AdamWHyper] = None, stream=None):
        self.params, self.hp = list(params), AdamWHyper() if hp is None else hp
        if not self.params:
            raise ValueError("params is empty")
        self.descs = [make_adamw_desc(p, self.hp) for p in self.params]
        self._dev = dev = self.params[0]["W"].device
        for p in self.params:
            if p["W"].device != dev:
                raise ValueError(f"W is on {p['W'].device}, expected {dev}")
        n = native.opt_adamw_workspace_size(self.descs)
        st = self._handle(stream)
        with torch.cuda.stream(stream):   # the table's: another stream may still write to what it hands out
            self.workspace = torch.empty(n, dtype=torch.uint8, device=dev)
        # what the table points to, whatever becomes of the dicts, and the streams that know of it
        self._held = [self.workspace, *(t for p in self.params for t in p.values() if isinstance(t, torch.Tensor))]
        self._streams = set()
        self._stream(stream)
        self._g = native.opt_adamw_create(self.descs, self.hp.c(), self.workspace.data_ptr(), n, st)

    def _handle(self, stream):
        dev = self._dev
        if dev.type != "cuda":
            raise ValueError("tensors must live on a HIP device")
        if dev.index != torch._C._cuda_getDevice():
            raise ValueError(f"tensors are on {dev}, which is not the current device (torch.cuda.device)")
        return torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream

    def _stream(self, stream):
        st = self._handle(stream)
        if st not in self._streams:   # no memory of the group is handed out again before this stream is past its calls
            for t in {t.untyped_storage().data_ptr(): t for t in self._held}.values():   # a flat buffer's parts once
                t.record_stream(torch.cuda.current_stream() if stream is None else stream)
            self._streams.add(st)
        return st

    def _scalar(self, t, name, dtype, stream):
        if t is None:
            return 0
        if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.numel() != 1 or t.device != self._dev:
            raise ValueError(f"{name} must be one {dtype} element on {self._dev}")
        if stream is not None:
            t.record_stream(stream)
        return t.data_ptr()

    def grad_norm(self, max_norm: float = float("inf"), stream=None) -> GradNorm:
        """The 2-norm of all gradients of the group together, and the factor
        min(1, max_norm / (norm + 1e-6)) for step's grad_scale."""
        st = self._stream(stream)
        if stream is None:
            out = torch.empty(2, device=self._dev)
        else:
            with torch.cuda.stream(stream):
                out = torch.empty(2, device=self._dev)
        p = out.data_ptr()
        native.opt_adamw_grad_norm(self._g, max_norm, p, p + 4, st)
        return GradNorm(*out.unbind())

    def step(self, grad_scale=None, rng: Optional[Rng] = None, device_step=None, stream=None):
        """One step. grad_scale: an fp32 scalar on the device that multiplies the
        gradients (where it is NaN, nothing is written; the group counts the step all the
        same: a program that does not want that sets t back, or counts in device_step).
        rng: the random bits that round 8-bit states; give each step another offset.
        device_step: an int64 scalar on the device that holds this step's number,
        counted from 1, for a replayed graph (else the group counts)."""
        st = self._stream(stream)
        bits = None
        if rng is not None:
            bits = rng.c()
            self._scalar(rng.device_offset, "device_offset", torch.int64, stream)
        native.opt_adamw_step(self._g, self._scalar(grad_scale, "grad_scale", torch.float32, stream), bits,
                              self._scalar(device_step, "device_step", torch.int64, stream), st)

    @property
    def t(self) -> int:
        return native.opt_adamw_get_step(self._g)

    @t.setter
    def t(self, value: int):
        native.opt_adamw_set_step(self._g, value)

    def set_lr(self, lr: float):
        native.opt_adamw_set_lr(self._g, lr)
        self.hp.lr = lr

    def __reduce__(self):   # two objects would free one handle
        raise TypeError("a group is not copied: make another group from its tensors, or copies of them, and set its t")

    def close(self):
        if getattr(self, "_g", None):
            native.opt_adamw_destroy(self._g)
            self._g = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
