"""Which stream an AdamWGroup takes its memory on, and which streams its tensors are
recorded on, with the library's calls and the allocator replaced (no GPU)."""

import contextlib

import pytest
import torch

from matrix_optimizer_step_02_amd import adamw


class Recorded(torch.Tensor):
    """A CPU tensor that says it is on the GPU, and notes the streams it is recorded on."""
    device = property(lambda self: torch.device("cuda", 0))

    def record_stream(self, stream):
        self.__dict__.setdefault("on", []).append(stream.cuda_stream)

    def __repr__(self):
        return "Recorded()"


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def tensor(n=300):
    return torch.zeros(n).as_subclass(Recorded)


@pytest.fixture
def device(monkeypatch):
    """A device whose current stream is ``now[-1]``; ``taken``: the streams that were current at each allocation."""
    class Device:
        now, taken = [Stream(10)], []

    @contextlib.contextmanager
    def on(stream):
        if stream is not None:
            Device.now.append(stream)
        yield
        if stream is not None:
            Device.now.pop()

    def empty(*size, dtype=None, device=None):
        Device.taken.append(Device.now[-1].cuda_stream)
        return torch.zeros(*size, dtype=dtype).as_subclass(Recorded)

    Device.now, Device.taken = [Stream(10)], []
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Device.now[-1])
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: Device.now[-1].cuda_stream, raising=False)
    monkeypatch.setattr(adamw, "make_adamw_desc", lambda p, hp: None)
    monkeypatch.setattr(adamw.native, "opt_adamw_workspace_size", lambda d: 512)
    monkeypatch.setattr(adamw.native, "opt_adamw_create", lambda *a: 0)
    monkeypatch.setattr(adamw.native, "opt_adamw_step", lambda *a: None)
    return Device


def param():
    return {k: tensor() for k in ("W", "G", "m", "v")}


@pytest.mark.parametrize("stream", [None, Stream(11)])
def test_the_workspace_is_taken_on_the_stream_that_fills_it(device, stream):
    """Memory handed out on another stream may have that stream's writes still to come, over the table."""
    adamw.AdamWGroup([param()], stream=stream)
    assert device.taken == [10 if stream is None else 11]


@pytest.mark.parametrize("stream", [None, Stream(11)])
def test_tensors_are_recorded_on_every_stream_that_steps_them(device, stream):
    """They may be from another stream's memory, the one the group was made on included."""
    p = param()
    made = 10 if stream is None else 11
    group = adamw.AdamWGroup([p], stream=stream)
    where = lambda: [t.__dict__.get("on", []) for t in (*p.values(), group.workspace)]  # noqa: E731
    assert where() == [[made]] * 5
    group.step(stream=stream)
    group.step(stream=Stream(12))
    group.step(stream=Stream(12))
    assert where() == [[made, 12]] * 5


def test_a_storage_is_recorded_once(device):
    """Tensors cut from one buffer."""
    parts = tensor(900).split(300)
    rest = [param() for _ in parts]
    adamw.AdamWGroup([p | {"W": x} for p, x in zip(rest, parts)])
    on = [x.__dict__.get("on", []) for x in parts]
    assert sorted(map(len, on)) == [0, 0, 1]
    on = [p["m"].__dict__.get("on", []) for p in rest]
    assert on == [[10]] * 3
