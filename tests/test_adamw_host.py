"""Host-side tests of the AdamW step: what include/matopt_adamw.h declares is
exported, and bad arguments are refused before the device is touched (no GPU)."""

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
    txt = open(os.path.join(ROOT, "include", "matopt_adamw.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    names = set(re.findall(r"\b(opt_adamw_[a-z0-9_]+)\s*\(", txt))
    assert names == set(N.EXPORTED_ADAMW)
    for name in names:
        assert hasattr(N.load(), name), name


def desc(N, at=0, bits=32, **kw):
    """1000 elements whose tensors are 1 MiB apart."""
    p = lambda k: BASE + (at << 24) + (k << 20)  # noqa: E731
    base = dict(n=1000, W=p(0), G=p(1), G_dtype=0, state_bits=bits, m=p(2), v=p(3), W16=p(6), W16_dtype=N.OPT_BF16,
                lr_scale=1.0, weight_decay=0.1)
    if bits == 8:
        base |= dict(m_scale=p(4), v_scale=p(5))
    return N.opt_adamw_desc(**(base | kw))


def hp(N, **kw):
    return N.opt_adamw_hparams(**(dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8) | kw))


def refused(N, status, fn, *args):
    with pytest.raises(N.MatoptError) as e:
        fn(*args)
    assert e.value.status == getattr(N, "OPT_" + status), str(e.value)
    assert len(str(e.value)) > 20


def create(N, descs, h=None, ws=BASE + (1 << 35), ws_bytes=1 << 20):
    return (N.opt_adamw_create, descs, h or hp(N), ws, ws_bytes, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), "EINVAL"), (dict(n=(1 << 35) + 1), "EUNSUPPORTED"), (dict(state_bits=16), "EUNSUPPORTED"),
    (dict(G_dtype=7), "EUNSUPPORTED"), (dict(W16_dtype=0), "EUNSUPPORTED"), (dict(lr_scale=-1.0), "EINVAL"),
    (dict(lr_scale=float("inf")), "EINVAL"), (dict(weight_decay=-0.1), "EINVAL"), (dict(weight_decay=float("nan")), "EINVAL"),
])
def test_descriptions_refused(N, kw, status):
    refused(N, status, N.opt_adamw_workspace_size, [desc(N), desc(N, 1, **kw)])
    refused(N, status, *create(N, [desc(N, **kw)]))


@pytest.mark.parametrize("bits", [32, 8])
def test_pointers_refused(N, bits):
    for key, each in (("W", 4), ("G", 4), ("m", bits // 8), ("v", bits // 8), ("m_scale", 4), ("v_scale", 4), ("W16", 2)):
        have = getattr(desc(N, bits=bits), key)
        if have is None:   # a scale of a state of 32 bits
            refused(N, "EINVAL", *create(N, [desc(N, bits=bits, **{key: BASE + (9 << 20)})]))
            continue
        if key != "W16":
            refused(N, "EINVAL", *create(N, [desc(N, bits=bits, **{key: 0})]))
        if each > 1:
            refused(N, "EINVAL", *create(N, [desc(N, bits=bits, **{key: have + 1})]))


@pytest.mark.parametrize("bits", [32, 8])
def test_overlaps_refused(N, bits):
    a = desc(N, bits=bits)
    keys = [k for k in ("W", "G", "m", "v", "m_scale", "v_scale", "W16") if getattr(a, k)]
    for k in keys:
        for other in keys:
            if k != other:   # within a tensor
                refused(N, "EINVAL", *create(N, [desc(N, bits=bits, **{k: getattr(a, other) + 4})]))
            if (k, other) != ("G", "G"):   # between two
                refused(N, "EINVAL", *create(N, [a, desc(N, 1, bits=bits, **{k: getattr(a, other) + 4})]))
    for k in keys:
        refused(N, "EINVAL", *create(N, [a], ws=getattr(a, k) // 256 * 256))
    # a small tensor inside a large gradient, behind another that ends before
    big = desc(N, 2, n=200000)
    refused(N, "EINVAL", *create(N, [big, desc(N, 3, n=10, G=big.G + 40), desc(N, 4, n=10, W=big.G + 400000)]))


def test_groups_refused(N):
    refused(N, "EINVAL", N.opt_adamw_workspace_size, [])
    ok = [desc(N, i, bits=(32, 8)[i % 2]) for i in range(3)]
    need = N.opt_adamw_workspace_size(ok)
    assert need % 256 == 0
    refused(N, "ENOWS", *create(N, ok, ws_bytes=need - 1))
    refused(N, "EINVAL", *create(N, ok, ws=0))
    refused(N, "EINVAL", *create(N, ok, ws=BASE + (1 << 35) + 64))
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(lr=float("inf")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
               dict(beta2=float("nan")), dict(eps=0.0), dict(eps=1e-60), dict(eps=float("inf"))):
        refused(N, "EINVAL", *create(N, ok, hp(N, **kw)))
    refused(N, "EUNSUPPORTED", *create(N, ok, hp(N, beta2=1 - 1e-12)))
    refused(N, "EUNSUPPORTED", N.opt_adamw_workspace_size, [desc(N, i, n=1 << 35) for i in range(2)])


def test_null_arguments_refused(N):
    lib, u, g, t = N.load(), C.c_uint64(0), C.c_void_p(0), C.c_int64(0)
    assert lib.opt_adamw_workspace_size(None, 1, C.byref(u)) == N.OPT_EINVAL
    assert lib.opt_adamw_workspace_size(desc(N), 1, None) == N.OPT_EINVAL
    assert lib.opt_adamw_create(desc(N), 1, None, BASE, 1 << 20, None, C.byref(g)) == N.OPT_EINVAL
    assert lib.opt_adamw_create(desc(N), 1, hp(N), BASE, 1 << 20, None, None) == N.OPT_EINVAL
    assert lib.opt_adamw_step(None, None, None, None, None) == N.OPT_EINVAL
    assert lib.opt_adamw_grad_norm(None, 1.0, BASE, BASE, None) == N.OPT_EINVAL
    assert lib.opt_adamw_grad_norm(None, 0.0, BASE, BASE, None) == N.OPT_EINVAL
    assert lib.opt_adamw_get_step(None, C.byref(t)) == N.OPT_EINVAL
    assert lib.opt_adamw_set_step(None, 3) == N.OPT_EINVAL
    assert lib.opt_adamw_set_lr(None, 3.0) == N.OPT_EINVAL
    lib.opt_adamw_destroy(None)


def test_tensors_are_checked_before_a_device_is_needed(N):
    import matrix_optimizer_step_02_amd as mo
    z = lambda n=300, dt=torch.float32: torch.zeros(n, dtype=dt)  # noqa: E731
    ok = {"W": z(), "G": z()} | mo.adamw_state(z())
    with pytest.raises(ValueError, match="HIP device"):
        mo.AdamWGroup([ok])
    with pytest.raises(ValueError, match="HIP device"):
        mo.AdamWGroup([{"W": z(), "G": z()} | mo.adamw_state(z(), 8)])
    for bad, match in [({"W": z(dt=torch.bfloat16)}, "W has dtype"), ({"G": z(dt=torch.float64)}, "G has dtype"),
                       ({"G": z(299)}, "G has shape"), ({"m": z(dt=torch.bfloat16)}, "m has dtype"),
                       ({"v": z(dt=torch.float8_e5m2)}, "v has dtype"), ({"W16": z()}, "W16 has dtype"),
                       ({"m_scale": z(2)}, "8 bits"), ({"W": torch.zeros(600)[::2]}, "contiguous"), ({"lr": 1.0}, "unknown"),
                       ({"m": z(dt=torch.float8_e4m3fn), "v": z(dt=torch.float8_e5m2), "m_scale": z(1), "v_scale": z(2)}, "m_scale")]:
        with pytest.raises(ValueError, match=match):
            mo.AdamWGroup([ok | bad])
    with pytest.raises(TypeError, match="m_scale"):
        mo.AdamWGroup([ok | {"m": z(dt=torch.float8_e4m3fn), "v": z(dt=torch.float8_e5m2)}])
    with pytest.raises(ValueError, match="empty"):
        mo.AdamWGroup([])
    with pytest.raises(ValueError, match="bits"):
        mo.adamw_state(z(), 4)
    with pytest.raises(AttributeError):
        mo.no_such_name
