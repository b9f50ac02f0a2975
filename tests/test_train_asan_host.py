"""The training-pass operators' host code under AddressSanitizer and UBSan.

Their sources are compiled with -fsanitize=address,undefined and no recovery
on the host side only (the device code is built as usual and never launched:
no GPU is touched), linked with tests/asan/train_driver.cpp, and run."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_optimizer_step_02_amd", "csrc")
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]


@pytest.mark.timeout(600)
def test_host_checks_are_clean_under_asan_and_ubsan(tmp_path):
    hipcc = next((c for c in ("/opt/rocm/bin/hipcc", shutil.which("hipcc")) if c and os.path.exists(c)), None)
    if hipcc is None:
        pytest.skip("hipcc not available")
    srcs = [os.path.join(CSRC, f) for f in ("attention.hip", "norm.hip", "policy_loss.hip")]
    srcs.append(os.path.join(ROOT, "tests", "asan", "train_driver.cpp"))
    common = ["-std=c++17", "-O1", "-g", "-fPIC", "--offload-arch=gfx950", "-I", os.path.join(ROOT, "include"),
              "-I", CSRC, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"] + SAN
    objs, procs = [], []
    for s in srcs:
        o = str(tmp_path / (os.path.basename(s) + ".o"))
        cmd = [hipcc, "-x", "hip"] + common + ["-c", s, "-o", o]
        procs.append((s, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
        objs.append(o)
    for s, p in procs:
        out, err = p.communicate()
        assert p.returncode == 0, f"compile {s}:\n{out}{err}"
    exe = str(tmp_path / "train_driver")
    r = subprocess.run([hipcc, "--offload-arch=gfx950", "-o", exe] + objs + SAN, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    env.pop("LD_PRELOAD", None)
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "0 failures" in r.stdout, r.stdout + r.stderr
    assert "AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr
