"""Packed rows in no sequence, before cu_seqlens[0] and from cu_seqlens[N] on: what they hold reaches no
result, and y and every gradient stay as they were there."""
import pytest
import torch

import gated_delta_rule_78_amd as kda
from gated_delta_rule_78_amd import glr as binding
from tests.parity import say
from tests.test_gpu_glr import BF16, F32, G_MIN, GUARD, check, kw, make, reference

pytestmark = pytest.mark.gpu

CASES = [
    # H, d, lens, rows before the first sequence, rows behind the last
    (2, 48, [70, 0, 300], 5, 3),
    (2, 48, [1], 255, 0),
    (3, 100, [0, 130, 1, 127, 0], 256, 90),       # a whole tile of rows in no sequence
    (1, 66, [700, 20], 700, 400),                 # more than one
    (2, 3, [60, 0, 200], 130, 140),               # a channel a thread
    (700, 7, [200, 0, 90], 300, 17),              # narrow heads side by side
    (2, 40, [0, 0], 300, 20),                     # no rows at all in a sequence
]
ids = lambda c: "%dx%d-%s-lead%d-tail%d" % (c[0], c[1], "+".join(map(str, c[2])), c[3], c[4]) if isinstance(c, tuple) else None


def build(case, dt, bad):
    H, d, lens, lead, tail = case
    c = make(0, H, 0, d, dt, lens=lens, z=True, u=True, s0=True, tail=lead + tail, seed=70)
    c["cu"] += lead
    end = lead + sum(lens)
    for k in ("x", "z", "u", "dy"):
        c[k][:, :lead] = bad
        c[k][:, end:] = bad
    inside = torch.zeros(c["T"], dtype=torch.bool, device=c["x"].device)
    inside[lead:end] = True
    return c, inside


def backward(c, dy, entry):
    """kda_glr_bwd into tensors that hold GUARD."""
    x = c["x"]
    full = lambda t: torch.full_like(t, GUARD)
    out = dict(dx=full(x), dd=full(x), du=full(x), dA=full(c["A"]), dS0=full(c["S0"]))
    desc = binding._desc(c["N"], c["H"], c["T"], c["d"], x.dtype, dy.dtype, True, "norm", G_MIN)
    gates = binding._gates(x, x.get_device(), x.shape, None, c["z"], c["A"], c["u"], c["H"], c["d"])
    lib = binding._library()
    ws = torch.empty(lib.kda_glr_bwd_workspace_bytes(desc, entry is not None, 1), dtype=torch.uint8, device=x.device)
    p = lambda t: None if t is None else t.data_ptr()
    st = lib.kda_glr_bwd(desc, p(x), gates, p(c["cu"]), p(c["S0"]), p(entry), p(dy), p(c["dS_T"]), p(out["dx"]), p(out["dd"]),
                         p(out["du"]), p(out["dA"]), p(out["dS0"]), p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_rows_outside(case, dt, bad):
    say("rows outside", ids(case), dt, bad)
    c, inside = build(case, dt, bad)
    y = torch.full_like(c["x"], GUARD)
    y, S_T, entry = kda.glr_fwd(c["x"], None, c["S0"], y=y, store_entry_states=True, **kw(c, "norm"))
    dy = c["dy"].to(dt)
    ref = reference(c, "norm", dy, c["dS_T"])
    check("y", y, ref["y"], dt)
    check("S_T", S_T, ref["S_T"], F32)
    assert bool((y[:, ~inside] == GUARD).all())
    for e in (entry, None):
        out = backward(c, dy, e)
        for k in ("dx", "dd", "du"):
            check(k, out[k], ref[k], dt)
            assert bool((out[k][:, ~inside] == GUARD).all()), k
        check("dA", out["dA"], ref["dA"], F32)
        check("dS0", out["dS0"], ref["dS0"], F32)
