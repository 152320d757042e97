"""The largest launches of the gated linear recurrence (no GPU): what would number 2^32 threads is
refused before any device work."""
import os
import shutil

import pytest

from tests.test_host_sanitizers import CSRC, NATIVE, ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_launches_past_32_bits_are_refused(tmp_path):
    exe = str(tmp_path / "glr_limits_check")
    out = _run(["g++", "-std=c++17"] + SAN + ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                                             "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                                             os.path.join(NATIVE, "glr_limits_check.cpp"),
                                             os.path.join(CSRC, "kda_glr_abi.cpp"), "-o", exe], exe)
    assert "glr limits check: ok" in out
