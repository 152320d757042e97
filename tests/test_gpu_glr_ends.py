"""The gated linear recurrence where fp32 ends: log decays down to the smallest normal number, where
w = sqrt(1 - alpha^2) is tiny and its derivative large."""
import pytest
import torch

import gated_delta_rule_78_amd as kda
from tests.parity import say
from tests.test_gpu_glr import F32, check, kw, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,T", [(2, 9), (2, 300)])
@pytest.mark.parametrize("scale", ["leaky", "norm"])
def test_log_decays_next_to_zero(scale, N, T):
    say("log decays next to zero", scale, N, T)
    c = make(N, 2, T, 12, F32, s0=True, seed=60)
    g = torch.Generator(device=c["x"].device).manual_seed(61)
    c["la"] = -(2.0 ** -(torch.rand(c["la"].shape, generator=g, device=c["x"].device) * 100 + 26)).contiguous()
    c["la"][..., 0] = -2.0 ** -126
    c["S0"] *= 2.0 ** -40                       # of the inputs' size, else they are lost in it
    y, S_T, entry = kda.glr_fwd(c["x"], c["la"], c["S0"], store_entry_states=True, **kw(c, scale))
    grads = kda.glr_bwd(c["x"], c["la"], c["S0"], c["dy"], c["dS_T"], entry_states=entry, **kw(c, scale))
    ref = reference(c, scale, c["dy"], c["dS_T"])
    check("y", y, ref["y"], F32)
    check("S_T", S_T, ref["S_T"], F32)
    for k, t in zip(("dx", "dd", "du", "dS0"), grads):
        if t is not None:
            check(k, t, ref[k], F32)
