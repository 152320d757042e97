"""States updated in place (S_T = S0) where a head's last channels would not fill a thread of their own
tile (d > 64 with d % 64 in 1, 2, 3), with more tiles than run at once."""
import pytest
import torch

import gated_delta_rule_78_amd as kda
from tests.parity import say
from tests.test_gpu_glr import BF16, F32, check, kw, make, reference

pytestmark = pytest.mark.gpu

# sequences or packed heads 513: the two tiles of a head's channels are up to 1023 workgroups apart
CASES = [
    # N, H, T, lens, dtype
    (513, 1, 200, None, F32),
    (171, 3, 600, None, BF16),       # three tiles a chain
    (0, 513, 0, [70, 0, 129, 1], F32),
    (0, 171, 0, [300, 0, 1, 299], BF16),
]
ids = lambda c: ("packed%d-%d" % (c[1], sum(c[3])) if c[3] else "%dx%dx%d" % c[:3]) if isinstance(c, tuple) else None


@pytest.mark.parametrize("d", [65, 66, 67, 129])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_states_in_place(case, d):
    N, H, T, lens, dt = case
    say("in place", ids(case), d)
    c = make(N, H, T, d, dt, lens=lens, z=True, u=True, s0=True, seed=40 + d)
    want = kda.glr_fwd(c["x"], None, c["S0"], store_entry_states=True, **kw(c, "norm"))
    S = c["S0"].clone()
    got = kda.glr_fwd(c["x"], None, S, S_T=S, store_entry_states=True, **kw(c, "norm"))
    torch.cuda.synchronize()
    assert got[1] is S
    for a, b, name in zip(got, want, ("y", "S_T", "entry states")):
        assert torch.equal(a, b), name
    ref = reference(c, "norm")
    check("y", got[0], ref["y"], dt)
    check("S_T", S, ref["S_T"], F32)


@pytest.mark.parametrize("d", [65, 67])
def test_resume_in_place(d):
    """A prefill in three parts, the state carried in place, is the prefill in one (to the bound)."""
    c = make(259, 1, 390, d, F32, z=True, u=True, s0=True, seed=50 + d)
    ref = reference(c, "leaky")
    S = c["S0"].clone()
    for a, b in ((0, 40), (40, 300), (300, 390)):
        cut = lambda t: t[:, :, a:b].contiguous()
        y, _, _ = kda.glr_fwd(cut(c["x"]), None, S, S_T=S, z=cut(c["z"]), A_log=c["A"], in_gate=cut(c["u"]),
                              input_scale="leaky")
        check("rows %d..%d" % (a, b), y, (ref["y"][0][:, :, a:b], ref["y"][1][:, :, a:b]), F32)
    check("S_T", S, ref["S_T"], F32)
