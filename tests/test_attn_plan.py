"""The bounds that the attention's workspace and launches rest on, over drawn and adversarial lengths (no GPU, under
AddressSanitizer and UndefinedBehaviorSanitizer)."""
import os
import shutil

import pytest

from tests.test_host_sanitizers import CSRC, NATIVE, ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_chunks_fit_the_workspace_and_the_launches(tmp_path):
    exe = str(tmp_path / "attn_plan_check")
    out = _run(["g++", "-std=c++17"] + SAN + ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                                             "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                                             os.path.join(NATIVE, "attn_plan_check.cpp"), "-o", exe], exe)
    assert "attention plan check: ok" in out
