"""The host-side checks of the attention operators built with AddressSanitizer
and UndefinedBehaviorSanitizer and run on the CPU: tests/sanitize/attn_driver.cpp
makes calls that return before the first HIP runtime call, so no GPU is needed.
Only host code is sanitized; the gfx950 device code is built as usual."""
import os

import pytest

from conftest import ROOT
from test_sanitizers import HERE, HIPCC, SAN_HOST, _clean_run, _run

SOURCES = ("k3moe_heads", "k3moe_attention", "k3moe_tree", "k3moe_logprobs")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_attention_host_checks_under_asan_and_ubsan(tmp_path):
    flags = [HIPCC, "-O1", "-g", "-std=c++17"] + SAN_HOST + ["-I", os.path.join(ROOT, "include")]
    objs = [str(tmp_path / (n + ".o")) for n in ("driver",) + SOURCES]
    r = _run(flags + ["-x", "c++", "-c", os.path.join(HERE, "attn_driver.cpp"), "-o", objs[0]])
    assert r.returncode == 0, r.stderr
    for name, o in zip(SOURCES, objs[1:]):
        src = os.path.join(ROOT, "mxfp4_routed_expert_sigmoid_amd", "csrc", name + ".hip")
        r = _run(flags + ["--offload-arch=gfx950", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
                          "-packed-fp32-ops", "-x", "hip", "-c", src, "-o", o])
        assert r.returncode == 0, r.stderr
    exe = str(tmp_path / "attn_asan")
    r = _run([HIPCC, "--offload-arch=gfx950"] + SAN_HOST + objs + ["-o", exe])
    assert r.returncode == 0, r.stderr
    _clean_run(exe)
