"""The tile geometry of the gated linear recurrence on the host (no GPU): no two tiles share a
channel, so that states updated in place are read and written by one workgroup alone."""
import os
import shutil

import pytest

from tests.test_host_sanitizers import CSRC, NATIVE, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_every_channel_has_one_tile(tmp_path):
    exe = str(tmp_path / "glr_tiles_check")
    out = _run(["g++", "-std=c++17"] + SAN + ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + CSRC,
                                             os.path.join(NATIVE, "glr_tiles_check.cpp"), "-o", exe], exe)
    assert "glr tiles check: ok" in out
