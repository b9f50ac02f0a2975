"""Host-side tests of attention's sinks (no GPU needed)."""

import numpy as np
import pytest

from oracle import train_ops as T
from tests.test_train_host import N, desc, refused  # noqa: F401


@pytest.mark.parametrize("kw", [dict(sinks=-1, window=4), dict(sinks=4), dict(sinks=4, causal=0)])
def test_refused(N, kw):  # noqa: F811
    refused(N, N.OPT_EINVAL, N.opt_attention_workspace_size, desc(N, **kw), 1)


@pytest.mark.parametrize("sinks", [0, 1, 64, 1 << 29, (1 << 31) - 1])
def test_any_number_goes(N, sinks):  # noqa: F811
    for window in (1, 100, 1 << 29, (1 << 31) - 1):
        for length in (1, 100, 1 << 20):
            N.opt_attention_workspace_size(desc(N, window=window, sinks=sinks, q_len=length, k_len=length), 1)


def test_the_oracles_mask():
    see = T.visible(4, 6, True, 2, 1)
    want = np.array([[1, 1, 1, 0, 0, 0], [1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]], dtype=bool)
    assert np.array_equal(see, want)
    assert np.array_equal(T.visible(9, 5, True, 3, 0), T.visible(9, 5, True, 3))
    assert np.array_equal(T.visible(7, 7, True, 2, 7), T.visible(7, 7, True))


@pytest.mark.parametrize("sinks", [-1, 1 << 31, 1 << 32])
def test_numbers_past_31_bits_are_refused(N, sinks):  # noqa: F811
    import torch
    from matrix_optimizer_step_02_amd import train
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="sinks"):
        train.attention_forward(x, x, x, causal=True, window=2, sinks=sinks)
