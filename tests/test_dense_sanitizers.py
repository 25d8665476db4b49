"""The host-side checks of the dense operators built with AddressSanitizer and
UndefinedBehaviorSanitizer and run on the CPU: tests/sanitize/dense_driver.cpp
makes calls that return before the first HIP runtime call, so no GPU is needed.
Only host code is sanitized; the gfx950 device code is built as usual."""
import os

import pytest

from conftest import ROOT
from test_sanitizers import HERE, HIPCC, SAN_HOST, _clean_run, _run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_dense_host_checks_under_asan_and_ubsan(tmp_path):
    inc = ["-I", os.path.join(ROOT, "include")]
    flags = [HIPCC, "-O1", "-g", "-std=c++17"] + SAN_HOST + inc
    objs = [str(tmp_path / n) for n in ("driver.o", "norm.o", "linear.o")]
    r = _run(flags + ["-x", "c++", "-c", os.path.join(HERE, "dense_driver.cpp"), "-o", objs[0]])
    assert r.returncode == 0, r.stderr
    for name, o in zip(("k3moe_norm.hip", "k3moe_linear.hip"), objs[1:]):
        src = os.path.join(ROOT, "mxfp4_routed_expert_sigmoid_amd", "csrc", name)
        r = _run(flags + ["--offload-arch=gfx950", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
                          "-packed-fp32-ops", "-x", "hip", "-c", src, "-o", o])
        assert r.returncode == 0, r.stderr
    exe = str(tmp_path / "dense_asan")
    r = _run([HIPCC, "--offload-arch=gfx950"] + SAN_HOST + objs + ["-o", exe])
    assert r.returncode == 0, r.stderr
    _clean_run(exe)
