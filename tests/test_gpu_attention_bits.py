"""GPU test that attention without sinks keeps its bits: digests of its results as they were before it took sinks, for
each kind of mask, layout and workgroup. (A change that is meant to change them, of the compiler's too, records new
ones: the other tests say whether they are right.)"""

import hashlib

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

CASES = {   # shapes, type, arguments, digest
    "window 77, 500 tokens": (
        dict(q=(1, 500, 4, 64), k=(1, 500, 2, 64)), "bf16", dict(causal=True, window=77), "0ab4f1dd201d5fe9"),
    "causal, 1100 tokens": (
        dict(q=(1, 1100, 4, 128), k=(1, 1100, 2, 128)), "bf16", dict(causal=True), "196723bd6ee79db0"),
    "causal, 40 sequences of 300": (
        dict(q=(40, 300, 16, 64), k=(40, 300, 16, 64)), "f16", dict(causal=True), "301cf0dd9dea8fed"),
    "no mask, 12 x 257 on 601": (
        dict(q=(12, 257, 8, 96), k=(12, 601, 4, 96)), "f16", dict(), "e689fb8bf91fd252"),
    "31 queries on 5000 keys, window 3000": (
        dict(q=(2, 31, 8, 128), k=(2, 5000, 2, 128)), "bf16", dict(causal=True, window=3000), "732f1dd4fa8c6d94"),
    "padded, heads of 40": (
        dict(q=(3, 200, 4, 40), k=(3, 180, 4, 40)), "bf16",
        dict(causal=True, q_lens=[200, 0, 77], k_lens=[180, 9, 64]), "635bbae6b8cc38fb"),
    "packed": (
        dict(q=(900, 8, 128), k=(900, 4, 128)), "bf16",
        dict(causal=True, window=130, start=[0, 300, 301, 301, 890], max=589), "690c66cf4899174c"),
    "packed, f16": (
        dict(q=(3000, 8, 64), k=(3000, 2, 64)), "f16", dict(causal=True, start=[3, 1300, 1364, 2990], max=1626), "ce8ca169d8b61d2d"),
}


def digest(name):
    from matrix_optimizer_step_02_amd import train
    shapes, dtype, how, _ = CASES[name]
    rng, how = np.random.default_rng(17), dict(how)
    mk = lambda s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).to(  # noqa: E731
        {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]).cuda()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, v, dout = mk(shapes["q"]), mk(shapes["k"]), mk(shapes["k"]), mk(shapes["q"])
    for n in ("q_lens", "k_lens"):
        if n in how:
            how[n] = ints(how[n])
    if "start" in how:
        start, most = ints(how.pop("start")), how.pop("max")
        how |= dict(q_start=start, k_start=start, max_q=most, max_k=most)
    out, lse = train.attention_forward(q, k, v, **how)
    grads = train.attention_backward(dout, q, k, v, out, lse, **how)
    torch.cuda.synchronize()
    h = hashlib.sha1()
    for t in (out, lse, *grads):
        h.update(t.contiguous().view(torch.uint8).cpu().numpy().tobytes())
    return h.hexdigest()[:16]


@pytest.mark.parametrize("name", CASES)
def test_bits(name):
    print("attention bits", name, flush=True)
    assert digest(name) == CASES[name][3]
