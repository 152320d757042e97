"""GPU parity of the block norms (kda_block_norm_fwd, kda_block_norm_bwd) with fp64. Every output
element is held to the bound that oracle.block_norm derives, plus half a step of its type."""
import numpy as np
import pytest
import torch

import gated_delta_rule_78_amd as kda
from oracle import block_norm
from tests.parity import host32, say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
TINY = {BF16: 2.0 ** -133, F32: 2.0 ** -149}


def make(rows, D, dt, rt, *, gate=True, residual=True, post=True, pre=True, lam=True, weights=True, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000 * seed + 7 * rows + D)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    c = dict(f=rn(rows, D).to(dt), x=(2.0 * rn(rows, D)).to(rt) if residual else None,
             gate=rn(rows, D).to(dt) if gate else None, w_post=1.0 + 0.1 * rn(D) if post and weights else None,
             lam=0.5 + 0.1 * rn(D) if lam else None, w_pre=1.0 + 0.1 * rn(D) if pre and weights else None,
             dxo=rn(rows, D).to(rt), dn=rn(rows, D).to(dt) if pre else None, post=post, pre=pre, rt=rt, dt=dt)
    return c


def kw(c, scale=0.7):
    return dict(gate=c["gate"], norm_weight=c["w_post"], post_norm=c["post"], eps=1e-6, scale=scale,
                scale_weight=c["lam"], pre_norm=c["pre"], pre_weight=c["w_pre"], pre_eps=1e-5)


def reference(c, scale=0.7, dxo=None, dn=None):
    h = lambda t: None if t is None else host32(t)
    scale, eps, pre_eps = (float(np.float32(v)) for v in (scale, 1e-6, 1e-5))   # what the C call receives
    return block_norm.evaluate(h(c["f"]), h(c["x"]), h(c["gate"]), h(c["w_post"]), h(c["lam"]), h(c["w_pre"]),
                               post=c["post"], pre=c["pre"], scale=scale, eps=eps, pre_eps=pre_eps, dxo=h(dxo), dn=h(dn))


def check(tag, got, ref, key, dt):
    val, bound = ref[key], ref[key + "_b"]
    g = host32(got).astype(np.float64)
    assert g.shape == val.shape, tag
    tol = bound + HALF_STEP[dt] * (np.abs(val) + bound) + TINY[dt]
    worst = float(np.max(np.abs(g - val) / tol)) if g.size else 0.0
    say("%s %s: worst error / bound %.3f" % (tag, key, worst))
    assert np.all(np.isfinite(g)) and worst <= 1.0, (tag, key)


CASES = [
    # rows, D, dtype, residual dtype, flags
    (1, 1, F32, F32, {}),
    (3, 16, BF16, F32, {}),
    (70, 128, BF16, BF16, dict(residual=False, pre=False, lam=False)),
    (17, 64, F32, F32, dict(gate=False)),
    (65, 63, BF16, BF16, {}),
    (9, 300, F32, BF16, dict(lam=False)),
    (33, 512, BF16, F32, dict(post=False)),
    (5, 520, BF16, BF16, dict(weights=False)),
    (6, 1001, F32, F32, dict(gate=False, post=False)),
    (4, 2048, BF16, BF16, {}),
    (3, 4095, BF16, F32, dict(residual=False)),
    (1200, 4096, BF16, BF16, {}),
    (7, 5000, F32, F32, dict(pre=False)),
    (2, 8192, BF16, BF16, {}),
    (3, 11111, BF16, BF16, {}),
    (3, 10001, F32, F32, {}),
    (2, 16384, F32, F32, {}),
    (3, 12000, BF16, F32, dict(gate=False)),
    # more rows than workgroups, rows off 8 elements
    (2501, 1001, BF16, BF16, {}),
    (40003, 65, BF16, F32, dict(lam=False)),
    (17000, 12, F32, BF16, {}),
    (1500, 2050, F32, F32, dict(pre=False)),
    (300, 8190, BF16, BF16, {}),
    (259, 9001, F32, F32, {}),
    (4, 16380, BF16, BF16, {}),
]
ids = lambda c: "%dx%d-%s-%s%s" % (c[0], c[1], "bf16" if c[2] == BF16 else "fp32", "bf16" if c[3] == BF16 else "fp32",
                                   "".join("-%s=%d" % kv for kv in c[4].items())) if isinstance(c, tuple) else None


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_forward(case):
    rows, D, dt, rt, flags = case
    c = make(rows, D, dt, rt, seed=1, **flags)
    say("block norm forward", ids(case))
    x_out, n = kda.block_norm_fwd(c["f"], c["x"], res_dtype=rt, **kw(c))
    torch.cuda.synchronize()
    ref = reference(c)
    check("fwd", x_out, ref, "x_out", rt)
    assert (n is None) == (not c["pre"])
    if n is not None:
        check("fwd", n, ref, "n", dt)


@pytest.mark.parametrize("which", ["both", "dx_out", "dn"])
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_backward(case, which):
    rows, D, dt, rt, flags = case
    c = make(rows, D, dt, rt, seed=2, **flags)
    dxo = c["dxo"] if which != "dn" else None
    dn = c["dn"] if which != "dx_out" else None
    if dxo is None and dn is None:
        pytest.skip("no pre-norm: there is no dn")
    say("block norm backward", ids(case), which)
    got = kda.block_norm_bwd(c["f"], c["x"], dxo, dn, **kw(c))
    torch.cuda.synchronize()
    ref = reference(c, dxo=dxo, dn=dn)
    types = dict(df=dt, dx=rt, dgate=dt, dw_post=F32, dlam=F32, dw_pre=F32)
    given = dict(df=True, dx=c["x"] is not None, dgate=c["gate"] is not None, dw_post=c["w_post"] is not None,
                 dlam=c["lam"] is not None, dw_pre=c["w_pre"] is not None)
    for key, t in zip(types, got):
        assert (t is not None) == given[key], key
        if t is None:
            continue
        if key == "dw_pre" and dn is None:
            assert not bool(t.any())
        else:
            check("bwd", t, ref, key, types[key])


@pytest.mark.parametrize("dt", [BF16, F32])
def test_bases_off_the_wide_alignment(dt):
    """Tensors that start one element into their storage give the same numbers to the bound."""
    rows, D = 5, 512
    c = make(rows, D, dt, dt, seed=7)

    def off(t):
        if t is None or t.dim() == 1:
            return t
        r = torch.empty(t.numel() + 1, device=DEV, dtype=t.dtype)[1:].view(t.shape)
        return r.copy_(t)

    o = {k: off(v) if torch.is_tensor(v) else v for k, v in c.items()}
    x_out, n = kda.block_norm_fwd(o["f"], o["x"], **kw(o))
    got = kda.block_norm_bwd(o["f"], o["x"], o["dxo"], o["dn"], **kw(o))
    ref = reference(c, dxo=c["dxo"], dn=c["dn"])
    check("off", x_out, ref, "x_out", dt)
    check("off", n, ref, "n", dt)
    for key, t in zip(("df", "dx", "dgate", "dw_post", "dlam", "dw_pre"), got):
        check("off", t, ref, key, dt if key[1:2] != "w" and key != "dlam" else F32)


def test_in_place_residual_and_its_gradient():
    c = make(300, 1024, BF16, F32, seed=3)
    want, n = kda.block_norm_fwd(c["f"], c["x"], **kw(c))
    x = c["x"].clone()
    got, n2 = kda.block_norm_fwd(c["f"], x, x_out=x, **kw(c))
    assert got is x and torch.equal(got, want) and torch.equal(n, n2)
    g1 = kda.block_norm_bwd(c["f"], c["x"], c["dxo"], c["dn"], **kw(c))
    d = c["dxo"].clone()
    g2 = kda.block_norm_bwd(c["f"], c["x"], d, c["dn"], dx=d, **kw(c))
    assert g2[1] is d and all(torch.equal(a, b) for a, b in zip(g1, g2))


def test_bad_rows_stay_alone():
    """A row of zeros, one of infinities and one of NaN change no other row."""
    c = make(20, 256, BF16, BF16, seed=4)
    want = kda.block_norm_fwd(c["f"], c["x"], **kw(c)) + kda.block_norm_bwd(c["f"], c["x"], c["dxo"], c["dn"], **kw(c))[:3]
    c["f"][3] = 0
    c["f"][5, 7] = float("inf")
    c["f"][9] = float("nan")
    got = kda.block_norm_fwd(c["f"], c["x"], **kw(c)) + kda.block_norm_bwd(c["f"], c["x"], c["dxo"], c["dn"], **kw(c))[:3]
    rest = [r for r in range(20) if r not in (3, 5, 9)]
    for a, b in zip(got, want):
        assert torch.equal(a[rest], b[rest])
        assert bool(torch.isfinite(a[3]).all()) and not bool(torch.isfinite(a[9]).any())


@pytest.mark.parametrize("D", [128, 100, 4096])
def test_no_rows(D):
    f, x, g = (torch.empty(0, D, device=DEV, dtype=BF16) for _ in range(3))
    w = torch.ones(D, device=DEV)
    x_out, n = kda.block_norm_fwd(f, x, gate=g, norm_weight=w, pre_weight=w)
    assert x_out.shape == n.shape == (0, D)
    out = kda.block_norm_bwd(f, x, x_out, n, gate=g, norm_weight=w, pre_weight=w)
    torch.cuda.synchronize()
    assert out[0].shape == (0, D) and not bool(out[3].any()) and not bool(out[5].any())


def test_offsets_past_32_bits():
    """Rows whose first element lies past 2^31: the same as those rows alone."""
    D = 8192
    rows = (1 << 31) // D + 100
    g = torch.Generator(device=DEV).manual_seed(4)
    base = torch.randn(1024, D, generator=g, device=DEV).to(BF16)
    f = base.repeat(-(-rows // 1024), 1)[:rows].contiguous()
    k = dict(scale=0.5, norm_weight=1.0 + 0.1 * torch.randn(D, generator=g, device=DEV), pre_norm=False)
    x_out, _ = kda.block_norm_fwd(f, f, **k)
    tail = f[-100:].contiguous()
    want, _ = kda.block_norm_fwd(tail, tail, **k)
    assert torch.equal(x_out[-100:], want)
    df = kda.block_norm_bwd(f, f, x_out, None, **k)[0]
    assert torch.equal(df[-100:], kda.block_norm_bwd(tail, tail, want, None, **k)[0])


def test_same_bits_and_captured_replay():
    c = make(2000, 1536, BF16, BF16, seed=5)
    run = lambda: kda.block_norm_fwd(c["f"], c["x"], **kw(c)) + kda.block_norm_bwd(c["f"], c["x"], c["dxo"], c["dn"], **kw(c))
    want = [t.clone() for t in run()]
    assert all(torch.equal(a, b) for a, b in zip(run(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(3):
        if i == 2:
            c["f"].mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        eager = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))


def test_gradients_against_differences():
    """Central differences of the forward itself in fp32 along random directions: the loss is
    sum(x_out * a) + sum(n * b) in fp64, the step h = 2^-6 of each input's size; the truncation is
    h^2 of third derivatives (of the size of the terms) and the cancellation 2^-24 / h of them."""
    c = make(8, 192, F32, F32, seed=6)
    grads = kda.block_norm_bwd(c["f"], c["x"], c["dxo"], c["dn"], **kw(c))
    h = 2.0 ** -6
    leaves = ["f", "x", "gate", "w_post", "lam", "w_pre"]
    for key, g in zip(leaves, grads):
        v = torch.randn(c[key].shape, generator=torch.Generator().manual_seed(1)).to(DEV)
        vals, mags = [], []
        for s in (1.0, -1.0):
            cc = dict(c)
            cc[key] = c[key] + s * h * v
            xo, n = kda.block_norm_fwd(cc["f"], cc["x"], **kw(cc))
            terms = torch.cat([(xo.double() * c["dxo"].double()).flatten(), (n.double() * c["dn"].double()).flatten()])
            vals.append(float(terms.sum()))
            mags.append(float(terms.abs().sum()))
        diff = (vals[0] - vals[1]) / (2 * h)
        want = float((g.double() * v.double()).sum())
        tol = mags[0] * (h * h * 4.0 + 2.0 ** -24 * 64 / h)
        say("%s: difference %.6f gradient %.6f tolerance %.4f" % (key, diff, want, tol))
        assert abs(diff - want) <= tol
