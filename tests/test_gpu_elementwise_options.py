"""What the C entries of the elementwise operators allow and the bindings do not ask for: gradients of
weights that are ones, outputs that are skipped; and every mix of the norms' types."""
import itertools

import numpy as np
import pytest
import torch

import gated_delta_rule_78_amd as kda
from gated_delta_rule_78_amd import block_norm as nb
from gated_delta_rule_78_amd import glr as gb
from oracle import block_norm
from tests.parity import host32, say
from tests.test_gpu_block_norm import check as check_norm
from tests.test_gpu_glr import BF16, F32, G_MIN, GUARD, kw, make

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
p = lambda t: None if t is None else t.data_ptr()
stream = lambda: torch.cuda.current_stream().cuda_stream


def norm_bwd(c, weights, wanted, dx=True):
    """kda_block_norm_bwd with `weights` given (a subset of w_post, lam, w_pre) and the gradients
    `wanted` of them written."""
    rows, D = c["f"].shape
    desc = nb._desc(rows, D, c["f"].dtype, c["x"].dtype, c["dn"].dtype, True, True, 0.5, 1e-6, 1e-6)
    lib = nb._library()
    w = [c[k] if k in weights else None for k in ("w_post", "lam", "w_pre")]
    out = dict(df=torch.empty_like(c["f"]), dgate=torch.empty_like(c["gate"]), dx=torch.empty_like(c["x"]) if dx else None)
    out.update({"d" + k: torch.full((D,), GUARD, device=DEV) for k in wanted})
    need = lib.kda_block_norm_bwd_workspace_bytes(desc)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    st = lib.kda_block_norm_bwd(desc, p(c["f"]), p(c["gate"]), p(c["x"]), *map(p, w), p(c["dxo"]), p(c["dn"]), p(out["df"]),
                                p(out["dgate"]), p(out["dx"]), *(p(out.get("d" + k)) for k in ("w_post", "lam", "w_pre")),
                                p(ws) if wanted else None, need if wanted else 0, stream())
    assert st == 0
    torch.cuda.synchronize()
    return out


def norm_case(rows, D, dt, seed=80):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    c = {k: rn(rows, D).to(dt) for k in ("f", "gate", "x", "dxo", "dn")}
    c.update({k: torch.ones(D, device=DEV) for k in ("w_post", "lam", "w_pre")})
    return c


@pytest.mark.parametrize("rows,D,dt", [(70, 128, BF16), (9, 1001, F32), (300, 4096, BF16), (5, 12288, F32)])
def test_gradients_of_weights_that_are_ones(rows, D, dt):
    """NULL weights are ones: their gradients are bit for bit those of weights of ones, together and alone."""
    c = norm_case(rows, D, dt)
    names = ("w_post", "lam", "w_pre")
    want = norm_bwd(c, names, names)
    for wanted in [names, ("w_post",), ("lam",), ("w_pre",), ()]:
        got = norm_bwd(c, (), wanted, dx=bool(wanted))
        for k, t in got.items():
            if t is not None:
                assert torch.equal(t, want[k]), (wanted, k)


@pytest.mark.parametrize("D", [72, 1001])
@pytest.mark.parametrize("ft,rt,nt", list(itertools.product([BF16, F32], repeat=3)))
def test_every_mix_of_types(D, ft, rt, nt):
    say("norm types", D, ft, rt, nt)
    c = norm_case(37, D, F32, seed=81)
    c.update({k: c[k].to(t) for k, t in (("f", ft), ("gate", ft), ("x", rt), ("dxo", rt), ("dn", nt))})
    k = dict(gate=c["gate"], norm_weight=c["w_post"], scale=0.5, scale_weight=c["lam"], pre_weight=c["w_pre"])
    x_out, n = kda.block_norm_fwd(c["f"], c["x"], out_dtype=nt, **k)
    assert x_out.dtype is rt and n.dtype is nt
    grads = kda.block_norm_bwd(c["f"], c["x"], c["dxo"], c["dn"], **k)
    eps = float(np.float32(1e-6))
    ref = block_norm.evaluate(*[host32(c[q]) for q in ("f", "x", "gate", "w_post", "lam", "w_pre")], post=True, pre=True,
                              scale=0.5, eps=eps, pre_eps=eps, dxo=host32(c["dxo"]), dn=host32(c["dn"]))
    for key, t, dt in zip(("x_out", "n", "df", "dx", "dgate", "dw_post", "dlam", "dw_pre"), (x_out, n) + grads,
                          (rt, nt, ft, rt, ft, F32, F32, F32)):
        assert t.dtype is dt
        check_norm("types", t, ref, key, dt)


@pytest.mark.parametrize("N,H,T,d,lens", [(3, 2, 9, 20, None), (2, 3, 600, 66, None), (0, 3, 0, 40, [300, 0, 1, 170])])
def test_states_that_are_not_wanted(N, H, T, d, lens):
    """S_T, entry states and dS0 skipped, S0 and dS_T left out: the other outputs do not change a bit."""
    c = make(N, H, T, d, BF16, lens=lens, z=True, u=True, s0=True, seed=82)
    dy = c["dy"].to(BF16)
    x = c["x"]
    y, S_T, entry = kda.glr_fwd(x, None, c["S0"], store_entry_states=True, **kw(c, "leaky"))
    y2, none, none2 = kda.glr_fwd(x, None, c["S0"], store_state=False, **kw(c, "leaky"))
    assert none is None and none2 is None and torch.equal(y, y2)
    zero = torch.zeros_like(c["S0"])
    assert all(torch.equal(a, b) for a, b in zip(kda.glr_fwd(x, None, None, **kw(c, "leaky"))[:2],
                                                kda.glr_fwd(x, None, zero, **kw(c, "leaky"))[:2]))
    want = kda.glr_bwd(x, None, c["S0"], dy, zero, entry_states=entry, **kw(c, "leaky"))
    got = kda.glr_bwd(x, None, c["S0"], dy, None, entry_states=entry, **kw(c, "leaky"))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    desc = gb._desc(c["N"], H, c["T"], d, BF16, BF16, lens is not None, "leaky", G_MIN)
    gates = gb._gates(x, x.get_device(), x.shape, None, c["z"], c["A"], c["u"], H, d)
    lib = gb._library()
    out = [torch.empty_like(x) for _ in range(3)] + [torch.empty_like(c["A"])]
    ws = torch.empty(lib.kda_glr_bwd_workspace_bytes(desc, 1, 1), dtype=torch.uint8, device=DEV)
    st = lib.kda_glr_bwd(desc, p(x), gates, p(c["cu"]), p(c["S0"]), p(entry), p(dy), None, *map(p, out), None, p(ws), ws.numel(),
                         stream())
    torch.cuda.synchronize()
    assert st == 0 and all(torch.equal(a, b) for a, b in zip(out, (want[0], want[1], want[2], want[4])))
