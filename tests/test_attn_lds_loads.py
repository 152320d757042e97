"""The attention's loads into LDS stand in inline assembly, before which the compiler keeps no waits: it has to know that
they write m0, and they have to wait for their scalar operands themselves (no GPU: the assembly of this tree's own
code is read)."""
import os
import re
import subprocess

import pytest

from gated_delta_rule_78_amd import build
from tests.test_host_sanitizers import NATIVE

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Instructions of each kernel of lds_load_check.hip, in order: (mnemonic, operands)."""
    out = str(tmp_path_factory.mktemp("asm") / "lds_load_check.s")
    r = subprocess.run([build.HIPCC] + build.COMMON + ["-S", "--offload-device-only", os.path.join(NATIVE, "lds_load_check.hip"),
                                                       "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert "clobber" not in r.stderr
    found, name = {}, None
    for line in open(out):
        label = re.match(r"_Z\d+(\w+?)(?:PK|Dv)\w*:", line)
        name = label[1] if label else name
        words = line.split(";")[0].split(None, 1)
        if name and words and re.match(r"[sv]_|buffer_|ds_|global_", words[0]):
            found.setdefault(name, []).append((words[0], words[1].strip() if len(words) > 1 else ""))
    return found


def registers(text):
    """The scalar registers that operands name."""
    return {r for a, b in re.findall(r"s\[(\d+):(\d+)\]", text) for r in range(int(a), int(b) + 1)} | {
        int(a) for a in re.findall(r"\bs(\d+)\b", text)}


def test_m0_is_set_again_behind_a_load(kernels):
    steps = [op if op != "s_mov_b32" else "m0" for op, args in kernels["lds_loads"]
             if op.startswith("buffer_load") or (op == "s_mov_b32" and args.startswith("m0"))]
    assert steps == ["m0", "buffer_load_dword", "m0", "buffer_load_dwordx4", "m0", "buffer_load_dword"]


def test_loads_wait_for_scalars_that_vector_instructions_wrote(kernels):
    """Five wait states between a lane read and a load that takes its result; an instruction is one, s_nop n n + 1."""
    code, loads = kernels["lane_descriptors"], 0
    for i, (op, args) in enumerate(code):
        if op != "buffer_load_dwordx4":
            continue
        loads += 1
        states, reads = 0, registers(args.split(",", 1)[1])
        for before, operands in reversed(code[:i]):
            if states >= 5:
                break
            assert not (before.startswith("v_read") and registers(operands.split(",")[0]) & reads), (states, before, operands)
            states += int(operands) + 1 if before == "s_nop" else 1
    assert loads
