"""Keys and values in one buffer: which layouts the append may take, against counting their elements (no GPU, under
AddressSanitizer and UndefinedBehaviorSanitizer)."""
import os
import shutil

import pytest

from tests.test_host_sanitizers import CSRC, NATIVE, ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_caches_of_unequal_widths_in_one_buffer(tmp_path):
    exe = str(tmp_path / "attn_layouts_check")
    out = _run(["g++", "-std=c++17"] + SAN + ["-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                                             os.path.join(NATIVE, "attn_layouts_check.cpp"), "-o", exe], exe)
    assert "attention layouts check: ok" in out
