"""GPU tests of 8-bit moments whose gradients differ widely within a block."""

import numpy as np
import pytest

from tests.test_adamw_spread import SPREADS, longest_step
from tests.test_gpu_adamw import HP, _mo, _torch, check, np64, param, snap

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spread", SPREADS)
@pytest.mark.parametrize("grad", ["f32", "bf16"])
def test_steps_stay_as_long_as_exact_moments_allow(spread, grad):
    """As the oracle's; the first steps to the bit, too. A weight is off by its own rounding, 2^-24 of at most 1."""
    torch, mo = _torch(), _mo()
    from matrix_optimizer_step_02_amd import train
    print(f"adamw spread {spread}, gradient {grad}", flush=True)
    p = param(700, 8, grad, seed=1)
    p["W"].zero_()
    mul = torch.from_numpy(np.resize(SPREADS[spread], 700)).cuda().float()
    hp = HP | dict(lr=2.0 ** -12, beta2=0.999)
    group = mo.AdamWGroup([p], mo.AdamWHyper(**hp))
    limit = 1.3 * max(longest_step(t, 0.9, 0.999) for t in (1, 2, 5, 10, 100, 1000))
    g = torch.Generator(device="cuda").manual_seed(2)
    for t in range(1, 301):
        p["G"].copy_(torch.randn(700, generator=g, device="cuda") * mul)
        before, w = snap(p) if t <= 20 else None, p["W"].clone()
        group.step(rng=train.Rng(5, t))
        torch.cuda.synchronize()
        if t <= 20:
            check(p, 0, before, t, (5, t), hp=hp)
        assert np.abs(np64(p["W"]) - np64(w)).max() <= limit * hp["lr"] + 2.0 ** -23, t
