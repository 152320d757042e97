"""The elementwise operators together with the KDA core, as a hybrid model runs them:
    n = pre-norm(x);  o = core(projections of n);  x, n = x + scale * gate * norm(o), pre-norm(x);  ...
Each operator of a run is held to its own oracle on the inputs it actually got (bounds derived in
oracle.glr and oracle.block_norm), and the ends of the run to the whole path in fp64."""
import numpy as np
import pytest
import torch

import gated_delta_rule_78_amd as kda
from gated_delta_rule_78_amd import synth
from oracle import backward, block_norm, gating, native
from tests.parity import TOL_O, assert_close, host32, say
from tests.test_gpu_bwd import check_grads
from tests.test_gpu_glr import check as check_glr
from tests.test_gpu_glr import reference as glr_reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
EPS = float(np.float32(1e-6))


def check_norm(tag, got, ref, dt):
    for key, t in got.items():
        val, bound = ref[key], ref[key + "_b"]
        err = np.abs(host32(t).astype(np.float64).reshape(val.shape) - val)
        tol = bound + HALF_STEP[dt] * (np.abs(val) + bound) + 2.0 ** -133
        worst = float(np.max(err / tol))
        say("%s %s: worst error / bound %.3f" % (tag, key, worst))
        assert worst <= 1.0, (tag, key)


def test_kda_output_gate_and_its_backward():
    """The core's fp32 output through block_norm is what the fused epilogue gives, and block_norm_bwd
    in front of chunk_bwd trains the gated core."""
    B, H, T, d = 1, 3, 200, 128
    q, k, v, la, beta, S0 = synth.prefill_inputs(B, H, T, d, d, BF16, device=DEV, seed_base=8100, s0_std=0.3)
    _, _, gate, w = synth.gating_inputs((B, H, T), H, d, d, BF16, device=DEV, seed=8101)
    o, _ = kda.chunk_fwd(q, k, v, la, beta, S0, out_dtype=F32)
    y, n = kda.block_norm_fwd(o, gate=gate.float(), norm_weight=w, pre_norm=False, res_dtype=BF16)
    assert n is None
    fused = kda.chunk_fwd_varlen(q, k, v, la, beta, None, S0, gate=gate, norm_weight=w, eps=1e-6)[0]
    # the same formula on the same fp32 core output: half a bf16 step each, and 2^-16 of the value for fp32
    diff = (y.float() - fused.float()).abs()
    tol = y.float().abs() * (2.0 ** -7 + 2.0 ** -16) + 1e-6
    say("epilogue against block_norm: worst %.3f of the tolerance" % float((diff / tol).max()))
    assert bool((diff <= tol).all())

    dy = torch.randn(B, H, T, d, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    dO, dx, dgate, dw, dlam, dpre = kda.block_norm_bwd(o, None, dy, None, gate=gate.float(), norm_weight=w, pre_norm=False)
    assert dx is None and dlam is None and dpre is None
    ref = block_norm.evaluate(host32(o), None, host32(gate), host32(w), None, None, post=True, pre=False, scale=1.0,
                              eps=EPS, pre_eps=EPS, dxo=host32(dy))
    check_norm("gate backward", {"df": dO, "dgate": dgate, "dw_post": dw}, ref, F32)
    got = kda.chunk_bwd(q, k, v, la, beta, S0, dO)
    f = lambda x: host32(x).reshape((B * H,) + tuple(x.shape[2:]))
    want = backward.kda_bwd(f(q), f(k), f(v), f(la), f(beta), f(S0), f(dO), None)
    check_grads("gated core", got, want, B * H)


def block(x, n, p, cu, S0, train):
    """One recurrent block on packed rows [T,D]: projections by matmul, everything else by the library."""
    proj = {k: (n @ p[k])[None] for k in ("wx", "wz", "wu")}          # [1,T,D]: one head of D channels
    g = n @ p["wg"]
    y, S_T, entry = kda.glr_fwd(proj["wx"], None, S0, z=proj["wz"], A_log=p["A"], in_gate=proj["wu"], input_scale="norm",
                                cu_seqlens=cu, store_entry_states=train)
    o = y[0] @ p["wo"]
    x2, n2 = kda.block_norm_fwd(o, x, gate=g, norm_weight=p["post"], scale=0.5, scale_weight=p["lam"], pre_weight=p["pre"])
    return x2, n2, S_T, dict(proj=proj, g=g, y=y, o=o, x=x, n=n, entry=entry)


def params(D, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    p = {k: (rn(D, D) / D ** 0.5).to(dtype) for k in ("wx", "wz", "wu", "wg", "wo")}
    p.update(A=torch.rand(1, D, generator=g, device=DEV) - 0.5, post=1 + 0.1 * rn(D), lam=1 + 0.1 * rn(D), pre=1 + 0.1 * rn(D))
    return p


def test_prefill_then_decode_of_a_block():
    """Prefill of a packed batch, then tokens one by one with the carried states: every operator
    against its oracle, and the decoded tokens against one longer prefill."""
    D, lens, more = 256, [130, 1, 299], 4
    p = params(D, BF16, 1)
    g = torch.Generator(device=DEV).manual_seed(2)
    xs = [torch.randn(n + more, D, generator=g, device=DEV).to(BF16) for n in lens]
    pre = lambda x: kda.block_norm_fwd(x, post_norm=False, pre_weight=p["pre"], store_x=False)[1]
    cu_of = lambda ls: torch.tensor(np.concatenate([[0], np.cumsum(ls)]), dtype=torch.int32, device=DEV)

    # the whole, in one go
    x_all = torch.cat(xs)
    whole, _, S_whole, t = block(x_all, pre(x_all), p, cu_of([n + more for n in lens]), None, False)
    ref = glr_reference(dict(N=3, H=1, T=len(x_all), d=D, cu=cu_of([n + more for n in lens]), x=t["proj"]["wx"], la=None,
                             z=t["proj"]["wz"], A=p["A"], u=t["proj"]["wu"], S0=None), "norm")
    check_glr("recurrence", t["y"], ref["y"], BF16)
    check_glr("states", S_whole, ref["S_T"], F32)
    rn = block_norm.evaluate(host32(t["o"]), host32(x_all), host32(t["g"]), host32(p["post"]), host32(p["lam"]),
                             host32(p["pre"]), post=True, pre=True, scale=0.5, eps=EPS, pre_eps=EPS)
    check_norm("block norm", {"x_out": whole}, rn, BF16)

    # prefill, then tokens: the projections of one row and of many may round differently (the matmul
    # adds in another order), by 2^-7 of the gates' inputs; the recurrence forgets them at its decay,
    # so outputs of size 1 agree to a few bf16 steps
    x_pre = torch.cat([x[:n] for x, n in zip(xs, lens)])
    _, _, S, _ = block(x_pre, pre(x_pre), p, cu_of(lens), None, False)
    starts = np.concatenate([[0], np.cumsum([n + more for n in lens])])[:-1]
    for i in range(more):
        x = torch.stack([x[n + i] for x, n in zip(xs, lens)])
        n = pre(x)
        proj = {k: (n @ p[k])[:, None] for k in ("wx", "wz", "wu")}   # [3,1,D]
        y = kda.glr_step(proj["wx"], None, S, z=proj["wz"], A_log=p["A"], in_gate=proj["wu"], input_scale="norm")
        x2, _ = kda.block_norm_fwd(y[:, 0] @ p["wo"], x, gate=n @ p["wg"], norm_weight=p["post"], scale=0.5,
                                   scale_weight=p["lam"], pre_weight=p["pre"])
        want = torch.stack([whole[s + m + i] for s, m in zip(starts, lens)])
        err = float((x2.float() - want.float()).abs().max())
        say("token %d: max |x - x_prefill| %.4f (values up to %.1f)" % (i, err, float(want.float().abs().max())))
        assert err <= 8 * 2.0 ** -8 * float(want.float().abs().max())
    err = float((S - S_whole).norm() / S_whole.norm())
    say("states after decode: rel-L2 %.2e" % err)
    assert err <= TOL_O[BF16]


def test_gradients_through_two_blocks():
    """fp32, two blocks: the chain of backward calls against fp64 automatic differentiation of the
    same path. Each of the path's operators is good to about 64 U32 and each matrix product of 96
    terms to 100 U32 of its terms' magnitude; two blocks chain 8 of each in either direction, and
    sums of D terms cancel to about 1 / sqrt(D) of that magnitude: 16 * 164 * 10 * 2^-24 = 1.6e-3
    of a gradient's norm."""
    D, lens = 96, [70, 0, 200, 1]
    T = sum(lens)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    ps = [params(D, F32, 10), params(D, F32, 11)]
    g = torch.Generator(device=DEV).manual_seed(12)
    x0 = torch.randn(T, D, generator=g, device=DEV)
    S0 = [torch.randn(len(lens), 1, D, generator=g, device=DEV) for _ in ps]
    da, db = torch.randn(T, D, generator=g, device=DEV), torch.randn(T, D, generator=g, device=DEV)
    first = 1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)

    x, n = kda.block_norm_fwd(x0, post_norm=False, pre_weight=first)
    tapes = []
    for p, s in zip(ps, S0):
        x, n, _, t = block(x, n, p, cu, s, True)
        tapes.append(t)
    grads = []
    dx, dn = da, db
    for p, s, t in reversed(list(zip(ps, S0, tapes))):
        do, dx, dg, dpost, dlam, dpre = kda.block_norm_bwd(t["o"], t["x"], dx, dn, gate=t["g"], norm_weight=p["post"],
                                                           scale=0.5, scale_weight=p["lam"], pre_weight=p["pre"])
        dy = (do @ p["wo"].t()).contiguous()[None]
        dxp, dzp, dup, dS0, dA = kda.glr_bwd(t["proj"]["wx"], None, s, dy, None, z=t["proj"]["wz"], A_log=p["A"],
                                             in_gate=t["proj"]["wu"], input_scale="norm", cu_seqlens=cu,
                                             entry_states=t["entry"])
        dn = dxp[0] @ p["wx"].t() + dzp[0] @ p["wz"].t() + dup[0] @ p["wu"].t() + dg @ p["wg"].t()
        nt = t["n"].t()
        grads.append(dict(post=dpost, lam=dlam, pre=dpre, wo=t["y"][0].t() @ do, wx=nt @ dxp[0], wz=nt @ dzp[0],
                          wu=nt @ dup[0], wg=nt @ dg, A=dA, S0=dS0))
    grads.reverse()
    dx0, _, _, _, _, dfirst = kda.block_norm_bwd(x0, None, dx, dn, post_norm=False, pre_weight=first)

    # the same path in fp64 with automatic differentiation
    leaf = lambda t: t.detach().cpu().double().requires_grad_()
    X0, F = leaf(x0), leaf(first)
    P = [{k: leaf(v) for k, v in dict(p, S0=s).items()} for p, s in zip(ps, S0)]
    rms = lambda v: v / (v.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    X, Nn = X0, rms(X0) * F
    for p in P:
        la = -5.0 * torch.sigmoid(torch.exp(p["A"]) * (Nn @ p["wz"]))
        a = torch.exp(la)
        b = (-torch.expm1(2 * la)).sqrt() * torch.sigmoid(Nn @ p["wu"]) * (Nn @ p["wx"])
        rows, at = [], 0
        for i, m in enumerate(lens):
            h = p["S0"][i, 0]
            for t in range(at, at + m):
                h = a[t] * h + b[t]
                rows.append(h)
            at += m
        o = torch.stack(rows) @ p["wo"]
        X = X + 0.5 * p["lam"] * torch.sigmoid(Nn @ p["wg"]) * rms(o) * p["post"]
        Nn = rms(X) * p["pre"]
    ((X * da.cpu().double()).sum() + (Nn * db.cpu().double()).sum()).backward()

    def rel(name, got, want):
        e = float((got.detach().cpu().double().reshape(want.shape) - want).norm() / want.norm())
        say("%s: rel-L2 %.2e" % (name, e))
        assert e <= 1.6e-3, name

    rel("x_out", x, X.detach())
    rel("dx0", dx0, X0.grad)
    rel("dfirst", dfirst, F.grad)
    for i, (gr, p) in enumerate(zip(grads, P)):
        for key, t in gr.items():
            rel("block %d d%s" % (i, key), t, p[key].grad)


def test_hybrid_layers_prefill():
    """A KDA layer and a recurrence layer over one residual stream, head-major rows between them."""
    B, H, T, d = 2, 2, 150, 64
    q, k, v, la, beta, S0 = synth.prefill_inputs(B, H, T, d, d, BF16, device=DEV, seed_base=8300, s0_std=0.2)
    o, S_T = kda.chunk_fwd(q, k, v, la, beta, S0)
    f = lambda x: host32(x).reshape((B * H,) + tuple(x.shape[2:]))
    o_ref, S_ref = native.kda_fwd(f(q), f(k), f(v), f(la), f(beta), f(S0))
    assert_close("core", BF16, f(o), o_ref, f(S_T), S_ref)
    x, n = kda.block_norm_fwd(o, v, gate=q, scale=0.5)
    y, S, _ = kda.glr_fwd(n, la, None, in_gate=k, input_scale="leaky")
    x2, n2 = kda.block_norm_fwd(y, x, gate=q, x_out=x)
    assert x2 is x
    ref = glr_reference(dict(N=B, H=H, T=T, d=d, cu=None, x=n, la=la, z=None, A=None, u=k, S0=None), "leaky")
    check_glr("recurrence", y, ref["y"], BF16)
    check_glr("states", S, ref["S_T"], F32)
    sig = gating.gated_rmsnorm(host32(o), host32(q), None, EPS)
    rn = block_norm.evaluate(host32(o), host32(v), host32(q), None, None, None, post=True, pre=True, scale=0.5, eps=EPS,
                             pre_eps=EPS)
    assert np.allclose(rn["x_out"], host32(v) + 0.5 * sig, atol=1e-12)
    check_norm("between", {"n": n}, rn, BF16)
