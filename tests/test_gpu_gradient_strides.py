"""GPU tests of gradients whose last axis is not contiguous, as autograd hands them over."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def strided(t, how):
    if how == "transposed":
        return t.transpose(-1, -2).contiguous().transpose(-1, -2)
    if how == "every second":
        wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], device=t.device, dtype=t.dtype)
        wide[..., ::2] = t
        return wide[..., ::2]
    return t[..., :1].expand_as(t)


@pytest.mark.parametrize("how", ["transposed", "every second", "expanded"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_of_any_strides(how, dtype):
    from matrix_optimizer_step_02_amd import train
    g = torch.Generator(device="cuda").manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    rope = train.Rotary(train.rotary_frequencies(48)[0])
    q, k = mk(2, 33, 6, 72), mk(2, 33, 2, 72)
    dyq, dyk = strided(mk(2, 33, 6, 72), how), strided(mk(2, 33, 2, 72), how)
    assert dyq.stride(-1) != 1 and dyk.stride(-1) != 1
    w = mk(72).float()
    *_, rq, rk = train.qk_norm_forward(q, k, w, w, rope=rope)
    for call in (lambda a, b: train.rotary_backward(a, b, rope, first=9),
                 lambda a, b: train.rotary_backward(a, None, rope, first=9)[:1],
                 lambda a, b: train.qk_norm_backward(a, b, q, k, w, w, rq, rk, rope=rope)):
        got, want = call(dyq, dyk), call(dyq.contiguous(), dyk.contiguous())
        assert all(torch.equal(x, y) and x.stride(-1) == 1 for x, y in zip(got, want))
        mixed = call(dyq, dyk.contiguous())
        assert all(torch.equal(x, y) for x, y in zip(mixed, want))
