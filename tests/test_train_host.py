"""Host-side tests of the training-pass operators: what include/matopt_train.h
declares is exported, and bad arguments are refused before the device is
touched (no GPU needed)."""

import ctypes as C
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 40


@pytest.fixture(scope="module")
def N():
    from matrix_optimizer_step_02_amd import native
    if not os.path.exists(native.LIB_PATH):
        pytest.skip("libmatopt.so not built (run __graft_entry__.build())")
    native.load()
    return native


def test_every_declared_symbol_is_exported(N):
    txt = open(os.path.join(ROOT, "include", "matopt_train.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    names = set(re.findall(r"\b(opt_[a-z0-9_]+)\s*\(", txt))
    assert names == set(N.EXPORTED_TRAIN)
    for name in names:
        assert hasattr(N.load(), name), name


def refused(N, status, fn, *args):
    with pytest.raises(N.MatoptError) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)
    assert len(str(e.value)) > 20


def desc(N, **kw):
    a = N.opt_attention_desc()
    base = dict(dtype=N.OPT_BF16, batch=2, heads=4, kv_heads=2, head_dim=64, q_len=8, k_len=8, causal=1, scale=0.125)
    for k, v in (base | kw).items():
        setattr(a, k, v)
    return a


def tensor(N, data=BASE, b=8 * 256, t=256, h=64):
    return N.opt_attention_tensor(data, b, t, h)


@pytest.mark.parametrize("kw,unsupported", [
    (dict(dtype=0), True), (dict(dtype=7), True), (dict(heads=3), False), (dict(heads=0), False),
    (dict(kv_heads=0), False), (dict(head_dim=0), False), (dict(head_dim=60), False), (dict(head_dim=136), True),
    (dict(q_len=-1), False), (dict(batch=-1), False), (dict(window=-1), False), (dict(window=4, causal=0), True),
    (dict(scale=0.0), False), (dict(scale=float("nan")), False), (dict(scale=float("inf")), False),
    (dict(q_start=BASE), False), (dict(q_start=BASE, k_start=BASE, q_lens=BASE), False),
    (dict(q_lens=BASE + 1), False), (dict(q_len=(1 << 30) + 1, k_len=8), True), (dict(batch=1 << 30, q_len=1 << 20), True),
    (dict(q_start=BASE, k_start=BASE, q_tokens=-1), False),
])
def test_attention_descriptions_refused(N, kw, unsupported):
    refused(N, N.OPT_EUNSUPPORTED if unsupported else N.OPT_EINVAL, N.opt_attention_workspace_size, desc(N, **kw), 1)


@pytest.mark.parametrize("kw,fits", [
    (dict(batch=1 << 25, heads=8, kv_heads=8, q_len=1, k_len=1), True),   # several launches
    (dict(q_len=1 << 29, k_len=1 << 29, heads=1, kv_heads=1, batch=1), True),
    (dict(q_len=(1 << 29) + 1, k_len=8, heads=1, kv_heads=1, batch=1), False),
    (dict(q_len=1 << 29, k_len=1 << 29, heads=64, kv_heads=8, batch=1), False),
])
def test_attention_limits(N, kw, fits):
    if fits:
        N.opt_attention_workspace_size(desc(N, **kw), 1)
    else:
        refused(N, N.OPT_EUNSUPPORTED, N.opt_attention_workspace_size, desc(N, **kw), 1)


@pytest.mark.parametrize("bad", [
    dict(data=0), dict(data=BASE + 8), dict(t=255), dict(h=60), dict(b=7), dict(t=-256),
])
def test_attention_tensors_refused(N, bad):
    a, ok = desc(N), tensor(N)
    for at in range(4):
        ts = [tensor(N, **bad) if i == at else ok for i in range(4)]
        refused(N, N.OPT_EINVAL, N.opt_attention_forward, a, *ts, BASE, 0, 0, 0)
    ws = N.opt_attention_workspace_size(a, 1)
    assert ws >= 2 * 8 * 4 * 4
    for at in range(8):
        ts = [tensor(N, **bad) if i == at else ok for i in range(8)]
        refused(N, N.OPT_EINVAL, N.opt_attention_backward, a, *ts[:5], BASE, *ts[5:], BASE, ws, 0)


def test_attention_outputs_and_workspace_refused(N):
    a, ok = desc(N), tensor(N)
    ws = N.opt_attention_workspace_size(a, 1)
    for bad in (dict(b=0), dict(t=0), dict(h=0), dict(t=8)):
        refused(N, N.OPT_EINVAL, N.opt_attention_forward, a, ok, ok, ok, tensor(N, **bad), BASE, 0, 0, 0)
    refused(N, N.OPT_EINVAL, N.opt_attention_forward, a, ok, ok, ok, ok, 0, 0, 0, 0)
    refused(N, N.OPT_EINVAL, N.opt_attention_forward, a, ok, ok, ok, ok, BASE + 2, 0, 0, 0)
    refused(N, N.OPT_ENOWS, N.opt_attention_backward, a, *[ok] * 5, BASE, *[ok] * 3, BASE, ws - 1, 0)
    refused(N, N.OPT_EINVAL, N.opt_attention_backward, a, *[ok] * 5, BASE, *[ok] * 3, 0, ws, 0)
    refused(N, N.OPT_EINVAL, N.opt_attention_backward, a, *[ok] * 5, BASE, *[ok] * 3, BASE + 16, ws, 0)
    refused(N, N.OPT_EUNSUPPORTED, N.opt_attention_forward, a, tensor(N, t=(1 << 24) + 8), ok, ok, ok, BASE, 0, 0, 0)


def test_null_arguments_refused(N):
    lib, u = N.load(), C.c_uint64(0)
    assert lib.opt_attention_workspace_size(None, 0, C.byref(u)) == N.OPT_EINVAL
    assert lib.opt_attention_workspace_size(desc(N), 0, None) == N.OPT_EINVAL
    assert lib.opt_attention_forward(desc(N), None, None, None, None, None, None, 0, None) == N.OPT_EINVAL
    assert lib.opt_layer_norm_workspace_size(4, 4, None) == N.OPT_EINVAL
    assert lib.opt_policy_loss_workspace_size(None, C.byref(u)) == N.OPT_EINVAL


def rng(N):
    return N.opt_rng(1, 2, 0)


@pytest.mark.parametrize("at,value,status", [
    (0, -1, "EINVAL"), (1, -1, "EINVAL"), (0, 1 << 32, "EUNSUPPORTED"), (1, 1 << 34, "EUNSUPPORTED"),
    (2, 5, "EUNSUPPORTED"), (3, 0, "EINVAL"), (3, BASE + 1, "EINVAL"), (4, 15, "EINVAL"), (6, 15, "EINVAL"),
    (7, 0, "EINVAL"), (8, 15, "EINVAL"), (9, -0.1, "EINVAL"), (9, 1.0, "EINVAL"), (9, float("nan"), "EINVAL"),
    (9, 0.999999, "EUNSUPPORTED"), (10, None, "EINVAL"),
])
def test_dropout_refused(N, at, value, status):
    args = [4, 16, N.OPT_F32, BASE, 16, BASE, 16, BASE, 16, 0.1, rng(N), 0]
    args[at] = value
    refused(N, getattr(N, "OPT_" + status), N.opt_dropout, *args)


@pytest.mark.parametrize("at,value,status", [
    (0, -1, "EINVAL"), (1, 0, "EINVAL"), (1, 16385, "EUNSUPPORTED"), (0, 1 << 31, "EUNSUPPORTED"),
    (2, 9, "EUNSUPPORTED"), (3, 0, "EINVAL"), (4, 15, "EINVAL"), (5, 2, "EUNSUPPORTED"), (7, 15, "EINVAL"),
    (8, 0, "EINVAL"), (8, BASE + 2, "EINVAL"), (9, BASE + 2, "EINVAL"), (10, -1.0, "EINVAL"), (11, 1.5, "EINVAL"),
    (12, None, "EINVAL"), (13, 0, "EINVAL"), (14, 3, "EINVAL"), (15, 0, "EINVAL"), (16, 3, "EINVAL"),
    (17, 0, "EINVAL"), (18, 0, "EINVAL"), (13, BASE + 1, "EINVAL"),
])
def test_layer_norm_forward_refused(N, at, value, status):
    args = [4, 16, N.OPT_BF16, BASE, 16, N.OPT_F32, BASE, 16, BASE, BASE, 1e-5, 0.1, rng(N), BASE, 16, BASE, 16, BASE,
            BASE, 0]
    args[at] = value
    refused(N, getattr(N, "OPT_" + status), N.opt_layer_norm_forward, *args)


def test_layer_norm_h_is_x_without_residual_and_dropout(N):
    refused(N, N.OPT_EINVAL, N.opt_layer_norm_forward, 4, 16, 0, BASE, 16, 0, 0, 0, BASE, 0, 1e-5, 0.0, None, BASE, 16,
            BASE, 16, BASE, BASE, 0)


@pytest.mark.parametrize("at,value,status", [
    (0, -1, "EINVAL"), (1, 0, "EINVAL"), (2, 9, "EUNSUPPORTED"), (3, 0, "EINVAL"), (4, 15, "EINVAL"),
    (5, 2, "EUNSUPPORTED"), (6, 0, "EINVAL"), (7, 15, "EINVAL"), (9, 15, "EINVAL"), (10, 0, "EINVAL"),
    (11, 0, "EINVAL"), (12, 0, "EINVAL"), (13, -1.0, "EINVAL"), (14, None, "EINVAL"), (15, 0, "EINVAL"),
    (16, 15, "EINVAL"), (18, 15, "EINVAL"), (19, 0, "EINVAL"), (20, BASE + 1, "EINVAL"), (21, 0, "EINVAL"),
    (21, BASE + 64, "EINVAL"), (22, 8, "ENOWS"),
])
def test_layer_norm_backward_refused(N, at, value, status):
    ws = N.opt_layer_norm_workspace_size(4, 16)
    args = [4, 16, N.OPT_BF16, BASE, 16, N.OPT_F32, BASE, 16, BASE, 16, BASE, BASE, BASE, 0.1, rng(N), BASE, 16, BASE,
            16, BASE, BASE, BASE, ws, 0]
    args[at] = value
    refused(N, getattr(N, "OPT_" + status), N.opt_layer_norm_backward, *args)


def policy(N, **kw):
    base = dict(dtype=N.OPT_F32, target_i64=0, rows=4, vocab=100, ld=100, logit_scale=1.0, clip_low=0.2, clip_high=0.2,
                kl_coef=0.1)
    return N.opt_policy_desc(**(base | kw))


@pytest.mark.parametrize("kw,unsupported", [
    (dict(dtype=4), True), (dict(rows=-1), False), (dict(vocab=0), False), (dict(rows=1 << 31), True),
    (dict(vocab=(1 << 31) - 1, ld=1 << 31), True), (dict(ld=99), False), (dict(logit_scale=0.0), False),
    (dict(logit_scale=float("nan")), False), (dict(clip_low=-0.1), False), (dict(clip_low=1.1), False),
    (dict(clip_high=-0.1), False), (dict(kl_coef=-1.0), False), (dict(kl_coef=float("nan")), False),
])
def test_policy_descriptions_refused(N, kw, unsupported):
    refused(N, N.OPT_EUNSUPPORTED if unsupported else N.OPT_EINVAL, N.opt_policy_loss_workspace_size, policy(N, **kw))


def test_policy_arguments_refused(N):
    a = policy(N)
    ws = N.opt_policy_loss_workspace_size(a)
    rows = N.opt_policy_rows(*[BASE] * 5)
    step = [a, BASE, rows, 1.0, BASE, BASE, BASE, 100, BASE, ws, 0]
    for at, value, status in [(1, 0, "EINVAL"), (1, BASE + 2, "EINVAL"), (2, None, "EINVAL"), (4, 0, "EINVAL"),
                              (5, BASE + 1, "EINVAL"), (6, 0, "EINVAL"), (7, 99, "EINVAL"), (7, 101, "EINVAL"),
                              (8, 0, "EINVAL"), (8, BASE + 8, "EINVAL"), (9, 1, "ENOWS")]:
        args = list(step)
        args[at] = value
        refused(N, getattr(N, "OPT_" + status), N.opt_policy_loss_step, *args)
    for i in range(5):
        r = N.opt_policy_rows(*[0 if i == j else BASE for j in range(5)])
        refused(N, N.OPT_EINVAL, N.opt_policy_loss_step, *step[:2], r, *step[3:])
        refused(N, N.OPT_EINVAL, N.opt_policy_loss_forward, a, BASE, r, BASE, BASE, BASE, BASE, BASE, ws, 0)
    for at in (1, 2, 3, 4, 6):
        args = [a, BASE, BASE, BASE, BASE, 0, BASE, 100, 0]
        args[at] = 0
        refused(N, N.OPT_EINVAL, N.opt_policy_loss_backward, *args)


def test_the_other_entry_points_still_refuse_half_precision(N):
    refused(N, N.OPT_EUNSUPPORTED, N.opt_gemm, 0, 0, 4, 4, 4, 1.0, BASE, N.OPT_F16, 4, BASE, 0, 4, 0.0, BASE, 4, 0)


def test_tensors_are_checked_before_a_device_is_needed(N):
    from matrix_optimizer_step_02_amd import train
    q, kv = torch.zeros(2, 8, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="HIP device"):
        train.attention_forward(q, kv, kv)
    with pytest.raises(ValueError, match="dtype"):
        train.attention_forward(q, kv, kv.float())
    with pytest.raises(ValueError, match="axes"):
        train.attention_forward(q[0], kv[0], kv[0])
    with pytest.raises(ValueError, match="come together"):
        train.attention_forward(q[0], kv[0], kv[0], q_start=torch.zeros(2, dtype=torch.int32))
    starts = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="max_q"):
        train.attention_forward(q[0], kv[0], kv[0], q_start=starts, k_start=starts)
    with pytest.raises(ValueError, match="q_lens"):
        train.attention_forward(q, kv, kv, q_lens=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="shape"):
        train.layer_norm_forward(torch.zeros(4, 8), torch.zeros(7))
    with pytest.raises(ValueError, match="dtype"):
        train.layer_norm_forward(torch.zeros(4, 8, dtype=torch.float64), torch.zeros(8))
    with pytest.raises(ValueError, match="rng"):
        train.layer_norm_forward(torch.zeros(4, 8), torch.zeros(8), p=0.5)
    with pytest.raises(ValueError, match="contiguous"):
        train.dropout(torch.zeros(8, 4).t(), 0.5, train.Rng(0))
    with pytest.raises(ValueError, match="device_offset"):
        train.dropout(torch.zeros(8, 4), 0.5, train.Rng(0, 0, torch.zeros(1)))
    v = torch.zeros(3)
    with pytest.raises(ValueError, match="ref_logp"):
        train.policy_loss_step(torch.zeros(3, 5), torch.zeros(3, dtype=torch.int64), v, v, v, kl_coef=0.1)
    with pytest.raises(ValueError, match="target"):
        train.policy_loss_step(torch.zeros(3, 5), v, v, v, v)


def test_policy_lse_rest_must_be_aligned(N):
    refused(N, N.OPT_EINVAL, N.opt_policy_loss_workspace_size, policy(N, lse_rest=BASE + 2))
    N.opt_policy_loss_workspace_size(policy(N, lse_rest=BASE + 4))


def test_policy_backward_takes_the_forward_calls_scale(N, monkeypatch):
    """The gradient is of the loss that was computed: its logit_scale comes with it, and another one is refused."""
    from matrix_optimizer_step_02_amd import train
    seen = []
    monkeypatch.setattr(train, "_stream", lambda dev: 0)
    monkeypatch.setattr(N, "opt_policy_loss_forward", lambda a, *rest: seen.append(a.logit_scale))
    monkeypatch.setattr(N, "opt_policy_loss_backward", lambda a, *rest: seen.append(a.logit_scale))
    x, t, v = torch.zeros(3, 5), torch.zeros(3, dtype=torch.int64), torch.zeros(3)
    f = train.policy_loss_forward(x, t, v, v, v, logit_scale=0.5)
    train.policy_loss_backward(x, t, f)
    train.policy_loss_backward(x, t, f, logit_scale=0.5)
    train.policy_loss_backward(x, t, f._replace(slope=2 * f.slope))
    assert seen == [0.5] * 4
    with pytest.raises(ValueError, match="logit_scale"):
        train.policy_loss_backward(x, t, f, logit_scale=1.0)
    del seen[:]
    four = train.PolicyForward(*f)   # of the four tensors alone
    train.policy_loss_backward(x, t, four)
    train.policy_loss_backward(x, t, four, logit_scale=0.5)
    assert seen == [1.0, 0.5]


def test_packed_outputs_whose_tokens_overlap_are_refused(N):
    """Sequences of one token share no row with each other either."""
    a = desc(N, batch=3, q_len=1, k_len=1, q_start=BASE, k_start=BASE, q_tokens=3, k_tokens=3)
    ok, bad, ws = tensor(N), tensor(N, t=0), N.opt_attention_workspace_size(a, 1)
    refused(N, N.OPT_EINVAL, N.opt_attention_forward, a, ok, ok, ok, bad, BASE, 0, 0, 0)
    for at in range(3):
        grads = [bad if n == at else ok for n in range(3)]
        refused(N, N.OPT_EINVAL, N.opt_attention_backward, a, *[ok] * 5, BASE, *grads, BASE, ws - 1, 0)


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Kernels are launched on the current device: its default stream has the same handle as every other device's."""
    from matrix_optimizer_step_02_amd import train
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 64 + index)
    assert train._stream(torch.device("cuda", 0)) == 64
    with pytest.raises(ValueError, match="current device"):
        train._stream(torch.device("cuda", 1))


def test_a_calls_tensors_are_recorded_on_its_stream(monkeypatch):
    """The allocator keeps their memory until that stream is done with it."""
    import contextlib

    from matrix_optimizer_step_02_amd import train
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    seen = []

    class Fake(torch.Tensor):
        is_cuda = True

        def record_stream(self, s):
            seen.append((int(self.numel()), s))

    mk = lambda n: torch.zeros(n).as_subclass(Fake)  # noqa: E731
    fwd = train.PolicyForward(mk(3), mk(4), mk(5), mk(6))
    fwd.lse_rest = mk(7)
    call = train._streamed(lambda *a, **kw: None)
    call(mk(1), 0.5, fwd, train.Rng(1, 2, mk(8)), out=mk(2), eps=1e-5, none=None, stream="s")
    assert sorted(seen) == [(n, "s") for n in range(1, 9)]
    del seen[:]
    call(mk(1), out=mk(2))   # on the current stream
    assert not seen


def test_tensors_that_require_a_gradient_are_refused_unless_gradients_are_off(N, monkeypatch):
    """There is no graph that would carry the gradient on: results that look whole would lose it."""
    from matrix_optimizer_step_02_amd import train
    monkeypatch.setattr(train, "_stream", lambda dev: 0)
    for name in ("opt_attention_forward", "opt_layer_norm_forward", "opt_dropout", "opt_policy_loss_forward"):
        monkeypatch.setattr(N, name, lambda *a: None)
    x, w, v = torch.zeros(3, 8), torch.zeros(8), torch.zeros(3)
    t, g = torch.zeros(3, dtype=torch.int64), lambda z: z.clone().requires_grad_()   # noqa: E731
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    calls = [lambda f: train.layer_norm_forward(f(x), w), lambda f: train.layer_norm_forward(x, f(w)),
             lambda f: train.layer_norm_forward(x, w, residual=f(x)), lambda f: train.dropout(f(x), 0.5, train.Rng(1)),
             lambda f: train.attention_forward(q, f(q), q), lambda f: train.policy_loss_forward(f(x), t, v, v, v)]
    for call in calls:
        call(lambda z: z)
        with pytest.raises(ValueError, match="gradient"):
            call(g)
        with torch.no_grad():
            call(g)


def test_a_step_counter_of_another_device_is_refused(N):
    """Kernels read it on the tensors' device."""
    from types import SimpleNamespace

    from matrix_optimizer_step_02_amd import train
    far = SimpleNamespace(dtype=torch.int64, numel=lambda: 1, device=torch.device("cuda", 1), data_ptr=lambda: BASE)
    with pytest.raises(ValueError, match="device_offset"):
        train.dropout(torch.zeros(4, 8), 0.5, train.Rng(0, 0, far))
    with pytest.raises(ValueError, match="device_offset"):
        train.layer_norm_forward(torch.zeros(4, 8), torch.zeros(8), p=0.5, rng=train.Rng(0, 0, far))
    with pytest.raises(ValueError, match="device_offset"):
        train.layer_norm_backward(torch.zeros(4, 8), torch.zeros(4, 8), torch.zeros(8), torch.zeros(4), torch.zeros(4),
                                  p=0.5, rng=train.Rng(0, 0, far))
