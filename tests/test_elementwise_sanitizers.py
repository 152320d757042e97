"""The validation layers of the gated linear recurrence and of the block norms under AddressSanitizer
and UndefinedBehaviorSanitizer (no GPU): host code over stub launchers, run as its own process."""
import os
import shutil

import pytest

from tests.test_host_sanitizers import CSRC, NATIVE, ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_elementwise_abi_under_sanitizers(tmp_path):
    exe = str(tmp_path / "elementwise_host_check")
    out = _run(["g++", "-std=c++17"] + SAN + ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                                             "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                                             os.path.join(NATIVE, "elementwise_host_check.cpp"),
                                             os.path.join(CSRC, "kda_glr_abi.cpp"), os.path.join(CSRC, "kda_norm_abi.cpp"),
                                             "-o", exe], exe)
    assert "elementwise host check: ok" in out
