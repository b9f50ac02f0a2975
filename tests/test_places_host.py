"""Which results may lie where: the overlaps of strided tensors against a walk over all elements, and the calls that
are refused for them (no GPU)."""

import os
import shutil
import subprocess

import pytest
import torch

from tests.test_heads_host import BASE, N, calls, desc, refused, rope, tensor  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_overlaps_are_those_of_the_elements(tmp_path):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "places")
    r = subprocess.run([cc, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I",
                        os.path.join(ROOT, "matrix_optimizer_step_02_amd", "csrc"), "-o", exe,
                        os.path.join(ROOT, "tests", "asan", "places_driver.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=100)
    assert r.returncode == 0 and r.stdout.startswith("0 wrong"), r.stdout + r.stderr


# q, k, yq, yk, dyq, dyk, dq, dk: each call's results and what it reads
RESULTS = {0: ((2, 3), (0, 1)), 1: ((2, 3), (0, 1)), 2: ((6, 7), (0, 1, 4, 5))}
OWN = {2: (0,), 3: (1,), 6: (0, 4), 7: (1, 5)}


@pytest.mark.skipif(torch.cuda.is_available(), reason="what is not refused would be launched")
@pytest.mark.parametrize("call", RESULTS)
def test_results_on_what_others_read_are_refused(N, call):  # noqa: F811
    d, r = desc(N, kv_heads=4), rope(N)
    far = [tensor(N, BASE + (i << 20)) for i in range(8)]
    for y in RESULTS[call][0]:
        for x in RESULTS[call][1]:
            for by in (0, 2, 256 * 2, 64 * 2):   # its place; an element, a token and a head further
                ts = list(far)
                ts[y] = tensor(N, ts[x].data + by)
                if by == 0 and x in OWN[y]:
                    continue
                refused(N, "EINVAL", *calls(N, d, r, ts)[call])
    a, b = RESULTS[call][0]
    for by in (0, 2, 256 * 2, 64 * 2):
        ts = list(far)
        ts[b] = tensor(N, ts[a].data + by)
        refused(N, "EINVAL", *calls(N, d, r, ts)[call])


@pytest.mark.skipif(torch.cuda.is_available(), reason="these would be launched")
@pytest.mark.parametrize("call", RESULTS)
def test_places_that_do_not_overlap_pass(N, call):  # noqa: F811
    """Views of one projection, in place and from one half of a buffer to the other: no GPU is what stops them."""
    d, r = desc(N), rope(N)
    wide = dict(b=8 * 1024, t=1024, h=64)
    q, k = tensor(N, **wide), tensor(N, BASE + 4 * 64 * 2, **wide)
    q2, k2 = tensor(N, BASE + 8 * 64 * 2, **wide), tensor(N, BASE + 12 * 64 * 2, **wide)
    other = [tensor(N, BASE + (i << 20)) for i in range(1, 5)]
    for ts in ([q, k, q, k, q2, k2, q, k], [q, k, q2, k2, *other[:2], q2, k2], [q, k, *other], [q, k, q, k, q2, k2, q2, k2]):
        if len(ts) == 6:
            ts = [*ts, *ts[2:4]]
        refused(N, "EHIP", *calls(N, d, r, ts)[call])
