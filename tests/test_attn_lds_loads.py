"""The attention's loads into LDS stand in inline assembly that writes m0: the compiler has to know, and to set m0 anew
for a load of its own behind one (no GPU: the assembly of this tree's own code is read)."""
import os
import re
import subprocess

import pytest

from gated_delta_rule_78_amd import build
from tests.test_host_sanitizers import NATIVE


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")
def test_m0_is_set_again_behind_a_load(tmp_path):
    out = str(tmp_path / "lds_load_check.s")
    r = subprocess.run([build.HIPCC] + build.COMMON + ["-S", "--offload-device-only", os.path.join(NATIVE, "lds_load_check.hip"),
                                                       "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    steps = re.findall(r"^\s+(s_mov_b32 m0|buffer_load_dword(?:x4)?)\b.*$", open(out).read(), re.M)
    assert steps == ["s_mov_b32 m0", "buffer_load_dword", "s_mov_b32 m0", "buffer_load_dwordx4", "s_mov_b32 m0", "buffer_load_dword"]
