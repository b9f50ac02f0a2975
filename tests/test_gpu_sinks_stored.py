"""GPU tests of sinks of so many sequences that a workgroup stores their gradients itself: more than 512 of sequences
times key heads, against the fp64 oracle as in test_gpu_sinks.py."""

import numpy as np
import pytest

from oracle import train_ops as T
from tests.test_gpu_attention import U, check_sequence, np64, run
from tests.test_gpu_sinks import _torch, dense, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sinks", [3, 40, 200])
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f16")])
def test_packed(sinks, d, dtype):
    """Sequences shorter and longer than the sinks, empty ones, tokens outside every sequence."""
    torch = _torch()
    print(f"sinks stored, packed, {sinks} sinks d {d}", flush=True)
    rng = np.random.default_rng(sinks)
    lens = [int(x) for x in rng.integers(0, 60, 300)]
    lens[7], lens[100], lens[-1] = 0, 900, 210
    n = sum(lens) + 5
    mk = normal(d, dtype)
    q, k, v, dout = mk(n, 4, d), mk(n, 2, d), mk(n, 2, d), mk(n, 4, d)
    st = torch.tensor(3 + np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    got = run(q, k, v, dout, causal=True, window=25, sinks=sinks, q_start=st, k_start=st, max_q=900, max_k=900)
    got = {x: np64(t) for x, t in got.items()}
    a = 3
    for m in lens:
        one = {x: got[x][a:a + m] for x in ("out", "dq", "dk", "dv")} | {"lse": got["lse"][:, a:a + m]}
        if m:
            check_sequence(np64(q[a:a + m]), np64(k[a:a + m]), np64(v[a:a + m]), np64(dout[a:a + m]), one, d ** -0.5,
                           T.visible(m, m, True, 25, sinks), U[dtype])
        a += m
    for x in ("out", "dq", "dk", "dv"):
        assert not got[x][:3].any() and not got[x][-2:].any(), x


@pytest.mark.parametrize("nq,nk", [(130, 130), (1, 90), (70, 40)])
def test_a_batch(nq, nk):
    dense(130, nq, nk, 8, 4, 32, 20, 33, seed=nq)
