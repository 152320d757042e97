"""GPU parity of the gated linear recurrence (kda_glr_fwd, kda_glr_bwd, kda_glr_step) with the fp64
token loop. Every output element is held to the bound that oracle.glr derives from counting fp32
roundings along its path, plus half a step of the output type."""
import numpy as np
import pytest
import torch

import gated_delta_rule_78_amd as kda
from oracle import glr
from tests.parity import host32, say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
TINY = {BF16: 2.0 ** -133, F32: 2.0 ** -149}    # a subnormal result is off by a whole step at most
G_MIN = -5.0
GUARD = 7.0


def make(N, H, T, d, dt, *, lens=None, z=False, u=False, s0=False, tail=0, seed=0, la_range=(-0.5, -0.001)):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17 * N + 31 * H + T + d)
    cu = None
    if lens is not None:
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
        N, T = len(lens), int(sum(lens)) + tail
    lead = (H, T) if lens is not None else (N, H, T)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    lo, hi = la_range
    c = dict(N=N, H=H, T=T, d=d, dt=dt, cu=cu, x=rn(*lead, d).to(dt), la=None, z=None, A=None, u=None, S0=None)
    if z:
        c["z"] = (rn(*lead, d) * 1.5 - 3.0).to(dt)
        c["A"] = torch.rand(H, d, generator=g, device=DEV) - 0.5
    else:
        c["la"] = (torch.rand(*lead, d, generator=g, device=DEV) * (lo - hi) + hi).to(dt)
    if u:
        c["u"] = rn(*lead, d).to(dt)
    if s0:
        c["S0"] = rn(N, H, d)
    c["dy"], c["dS_T"] = rn(*lead, d), rn(N, H, d)
    return c


def kw(c, scale):
    return dict(z=c["z"], A_log=c["A"], g_min=G_MIN, in_gate=c["u"], input_scale=scale, cu_seqlens=c["cu"])


def reference(c, scale, dy=None, dS_T=None):
    """fp64 outputs and bounds: dict name -> (value, bound), rows in no sequence NaN."""
    shape, sshape = tuple(c["x"].shape), (c["N"], c["H"], c["d"])
    host = {k: (None if c[k] is None else host32(c[k]).astype(np.float64)) for k in ("x", "la", "z", "A", "u", "S0")}
    ref = {k: (np.full(shape, np.nan), np.full(shape, np.nan)) for k in ("y", "dx", "dd", "du")}
    ref.update({k: (np.zeros(sshape), np.zeros(sshape)) for k in ("S_T", "dS0")})
    ref["dA"] = (np.zeros(sshape[1:]), np.zeros(sshape[1:]))
    zero = np.zeros(c["d"])
    cu = None if c["cu"] is None else c["cu"].cpu().numpy()
    for n, h, at in glr.sequences(c["N"], c["H"], c["T"], cu):
        part = lambda k: None if host[k] is None else host[k][at]
        q = glr.gates(part("x"), part("la"), part("z"), None if host["A"] is None else host["A"][h], G_MIN, part("u"), scale)
        s0 = zero if host["S0"] is None else host["S0"][n, h]
        hs, prev, last = glr.forward(q, s0)
        hb, lb = glr.forward_bound(q, s0, scale)
        ref["y"][0][at], ref["y"][1][at] = hs, hb
        ref["S_T"][0][n, h], ref["S_T"][1][n, h] = last, lb
        if dy is None:
            continue
        dyr = host32(dy).astype(np.float64)[at]
        ds = zero if dS_T is None else host32(dS_T).astype(np.float64)[n, h]
        r = glr.backward(q, prev, dyr, ds, G_MIN)
        b = glr.backward_bounds(q, prev, hb, dyr, ds, scale, s0, G_MIN)
        for k in ("dx", "dd") + (("du",) if host["u"] is not None else ()):
            ref[k][0][at], ref[k][1][at] = r[k], b[k]
        ref["dS0"][0][n, h], ref["dS0"][1][n, h] = r["dS0"], b["dS0"]
        if host["z"] is not None:
            ref["dA"][0][h] += r["dA"]
            ref["dA"][1][h] += b["dA"]
    return ref


def check(tag, got, ref, dt):
    """Every element within its bound plus half a step of its type; where the reference is NaN
    (rows in no sequence), the element is not looked at."""
    val, bound = ref
    g = host32(got).astype(np.float64)
    assert g.shape == val.shape, tag
    if g.size == 0:
        return
    ok = ~np.isnan(val)
    tol = bound + HALF_STEP[dt] * (np.abs(val) + bound) + TINY[dt]
    err = np.abs(g - val)
    worst = float(np.max(np.where(ok, err / tol, 0.0)))
    say("%s: worst error / bound %.3f" % (tag, worst))
    assert np.all(np.isfinite(g[ok])) and worst <= 1.0, tag


def run_fwd(c, scale, odt):
    y = torch.full(tuple(c["x"].shape), GUARD, device=DEV, dtype=odt)
    y, S_T, entry = kda.glr_fwd(c["x"], c["la"], c["S0"], out_dtype=odt, y=y, store_entry_states=True, **kw(c, scale))
    torch.cuda.synchronize()
    return y, S_T, entry


CASES = [
    # (N, H, T, d, lens), dtype, out dtype, z, u, scale, S0
    ((1, 1, 1, 1, None), BF16, BF16, False, False, "one", False),
    ((2, 3, 2, 3, None), F32, F32, True, True, "norm", True),
    ((1, 2, 255, 64, None), BF16, F32, False, True, "leaky", True),
    ((1, 2, 256, 8, None), F32, BF16, True, False, "one", False),
    ((2, 2, 257, 128, None), BF16, BF16, True, True, "norm", True),
    ((3, 1, 777, 77, None), F32, F32, False, False, "one", True),
    ((1, 3, 1300, 40, None), BF16, BF16, False, True, "norm", False),
    ((1, 1, 600, 300, None), F32, F32, True, True, "leaky", False),
    ((2, 1, 33, 1001, None), BF16, BF16, True, False, "norm", True),
    ((0, 2, 0, 64, [3, 0, 300, 1, 256, 0]), BF16, BF16, True, True, "norm", True),
    ((0, 3, 0, 100, [0, 0, 1000, 1, 500]), F32, F32, False, False, "leaky", True),
    ((0, 1, 0, 72, [1] * 40), BF16, F32, True, False, "one", False),
    ((0, 2, 0, 5, [255, 1, 256, 257, 2, 510]), F32, F32, False, True, "norm", False),
    ((0, 1, 0, 16, [0, 0, 0]), F32, F32, False, False, "one", True),
    # many chains of tiles (the others have few)
    ((2, 40, 600, 68, None), BF16, BF16, True, True, "norm", True),
    ((0, 70, 0, 20, [300, 0, 7, 500]), F32, F32, True, False, "leaky", True),
    # sequences short enough for a thread per channel, aligned and not; long ones with channels enough
    ((40, 3, 16, 36, None), BF16, BF16, True, True, "norm", True),
    ((70, 2, 9, 11, None), F32, BF16, False, True, "leaky", True),
    ((33, 1, 5, 64, None), F32, F32, True, False, "one", False),
    ((5, 1, 17, 20, None), BF16, F32, False, False, "norm", True),
    ((1, 2, 18, 131072, None), BF16, BF16, True, True, "norm", True),
    # narrow heads, several in a tile (1024 tiles and more): the last tile's places not all taken,
    # channels off 4; dA_log from many parts
    ((49, 7, 300, 8, None), BF16, BF16, True, True, "norm", True),
    ((180, 3, 260, 20, None), F32, F32, False, True, "leaky", True),
    ((1030, 1, 17, 31, None), BF16, F32, True, False, "one", False),
    ((55, 19, 20, 4, None), BF16, BF16, False, True, "norm", True),
    ((0, 513, 0, 9, [55, 0, 200, 1, 100]), F32, BF16, True, True, "leaky", True),
    ((0, 515, 0, 7, [3, 400]), BF16, BF16, False, False, "norm", False),
    ((0, 3, 0, 32, [130, 1, 126]), F32, F32, True, True, "norm", True),
    ((1, 1, 300, 12, None), BF16, BF16, True, False, "norm", True),
    ((700, 2, 3, 5, None), F32, F32, True, True, "norm", True),
    # more chains than tile counters, no multiple of the XCDs
    ((1, 1, 260, 66010, None), BF16, BF16, True, True, "norm", True),
    # a chain longer than any look back
    ((1, 1, 6000, 8, None), F32, F32, False, True, "leaky", True),
]


def build(case, seed=1, tail=0):
    (N, H, T, d, lens), dt, odt, z, u, scale, s0 = case
    c = make(N, H, T, d, dt, lens=lens, z=z, u=u, s0=s0, tail=tail if lens is not None else 0, seed=seed)
    return c, scale, dt, odt


def name(case):
    (N, H, T, d, lens), dt, odt, z, u, scale, s0 = case
    return "%s-%s-%s%s%s" % ("packed%d" % sum(lens) if lens is not None else "%dx%dx%d" % (N, H, T), d,
                             "bf16" if dt == BF16 else "fp32", "-z" if z else "", "-u" if u else "") + "-" + scale


@pytest.mark.parametrize("case", CASES, ids=name)
def test_forward(case):
    c, scale, dt, odt = build(case)
    say("forward", name(case))
    y, S_T, entry = run_fwd(c, scale, odt)
    ref = reference(c, scale)
    check("y", y, ref["y"], odt)
    check("S_T", S_T, ref["S_T"], F32)
    # entry states: the state before row c * GLR_CHUNK of its block of rows
    if c["cu"] is None and c["T"] > kda.GLR_CHUNK:
        val, bound = ref["y"]
        rows = np.arange(kda.GLR_CHUNK, c["T"], kda.GLR_CHUNK) - 1
        shape = (c["N"] * c["H"], len(rows), c["d"])
        check("entry states", entry[:, 1:], (val[:, :, rows].reshape(shape), bound[:, :, rows].reshape(shape)), F32)


@pytest.mark.parametrize("with_entry", [True, False])
@pytest.mark.parametrize("case", CASES, ids=name)
def test_backward(case, with_entry):
    c, scale, dt, odt = build(case, seed=2)
    say("backward", name(case), "entry states given" if with_entry else "recomputed")
    dy = c["dy"].to(odt)
    dS_T = c["dS_T"] if case[-1] else None
    entry = run_fwd(c, scale, odt)[2] if with_entry else None
    dx, dd, du, dS0, dA = kda.glr_bwd(c["x"], c["la"], c["S0"], dy, dS_T, entry_states=entry, **kw(c, scale))
    torch.cuda.synchronize()
    ref = reference(c, scale, dy, dS_T)
    check("dx", dx, ref["dx"], dt)
    check("ddecay", dd, ref["dd"], dt)
    check("dS0", dS0, ref["dS0"], F32)
    assert (du is None) == (c["u"] is None) and (dA is None) == (c["z"] is None)
    if du is not None:
        check("din_gate", du, ref["du"], dt)
    if dA is not None:
        check("dA_log", dA, ref["dA"], F32)


@pytest.mark.parametrize("N,H,d,dt,odt,z,u,scale", [
    (1, 1, 1, BF16, BF16, False, False, "one"),
    (1, 32, 128, BF16, BF16, True, True, "norm"),
    (5, 3, 77, F32, F32, False, True, "leaky"),
    (64, 4, 40, BF16, F32, True, False, "leaky"),
    (7, 2, 1001, F32, BF16, False, False, "norm"),
])
def test_step_chain(N, H, d, dt, odt, z, u, scale):
    """Six tokens through glr_step give the forward's outputs, the state carried in place."""
    T = 6
    c = make(N, H, T, d, dt, z=z, u=u, s0=True, seed=3)
    ref = reference(c, scale)
    S = c["S0"].clone()
    cut = lambda t, i: None if t is None else t[:, :, i].contiguous()
    for i in range(T):
        y = kda.glr_step(cut(c["x"], i), cut(c["la"], i), S, z=cut(c["z"], i), A_log=c["A"], g_min=G_MIN,
                         in_gate=cut(c["u"], i), input_scale=scale, out_dtype=odt)
        check("step %d" % i, y, (ref["y"][0][:, :, i], ref["y"][1][:, :, i]), odt)
    check("S", S, ref["S_T"], F32)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_bases_off_the_wide_alignment(dt):
    """Tensors that start one element into their storage."""
    c = make(1, 3, 300, 64, dt, z=True, u=True, s0=True, seed=12)

    def off(t):
        r = torch.empty(t.numel() + 1, device=DEV, dtype=t.dtype)[1:].view(t.shape)
        return r.copy_(t)

    o = {k: off(v) if torch.is_tensor(v) else v for k, v in c.items()}
    y, S_T, entry = kda.glr_fwd(o["x"], None, o["S0"], y=off(torch.zeros_like(o["x"])), S_T=off(torch.zeros_like(o["S0"])),
                                store_entry_states=True, **kw(o, "norm"))
    dy = off(c["dy"].to(dt))
    grads = kda.glr_bwd(o["x"], None, o["S0"], dy, o["dS_T"], entry_states=entry, **kw(o, "norm"))
    ref = reference(c, "norm", dy, c["dS_T"])
    check("y", y, ref["y"], dt)
    check("S_T", S_T, ref["S_T"], F32)
    for k, g in zip(("dx", "dd", "du", "dS0", "dA"), grads):
        check(k, g, ref[k], F32 if k in ("dS0", "dA") else dt)
    S = o["S0"].clone()
    one = lambda k: off(c[k][:, :, 0])
    ys = kda.glr_step(one("x"), None, S, z=one("z"), A_log=o["A"], g_min=G_MIN, in_gate=one("u"), input_scale="norm")
    check("step", ys, (ref["y"][0][:, :, 0], ref["y"][1][:, :, 0]), dt)


def test_rows_behind_the_last_sequence_stay():
    lens = [70, 300]
    c = make(0, 2, 0, 48, F32, lens=lens, z=True, u=True, s0=True, tail=90, seed=4)
    for k in ("x", "z", "u"):                       # what lies there must not matter
        c[k][:, 370:] = float("nan")
    y, S_T, entry = run_fwd(c, "norm", F32)
    ref = reference(c, "norm", c["dy"], c["dS_T"])
    check("y", y, ref["y"], F32)
    check("S_T", S_T, ref["S_T"], F32)
    assert bool((y[:, 370:] == GUARD).all())
    dy = c["dy"].clone()
    dy[:, 370:] = float("nan")
    grads = kda.glr_bwd(c["x"], None, c["S0"], dy, c["dS_T"], entry_states=entry, **kw(c, "norm"))
    for k, g in zip(("dx", "dd", "du", "dS0", "dA"), grads):
        check(k, g, ref[k], F32)


def test_packed_states_in_place():
    """S_T in place of S0, sequences that start and end inside a tile, over tiles, and empty ones."""
    c = make(0, 2, 0, 203, F32, lens=[0, 5, 3, 1, 0, 900, 127, 1, 300, 0], z=True, u=True, s0=True, seed=13)
    ref = reference(c, "norm")
    S = c["S0"].clone()
    y, S_T, _ = kda.glr_fwd(c["x"], None, S, S_T=S, **kw(c, "norm"))
    assert S_T is S
    check("y", y, ref["y"], F32)
    check("S_T", S, ref["S_T"], F32)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_packed_equals_sequences_alone(dt):
    """A packed batch gives what each sequence alone gives, to the bound of both: no state leaks
    over a boundary, not even a non-finite one."""
    lens = [300, 5, 256, 0, 190]
    c = make(0, 2, 0, 64, dt, lens=lens, u=True, seed=5)
    c["x"][:, 100] = float("inf")                   # sequence 0 from its row 100 on
    y, S_T, _ = run_fwd(c, "leaky", F32)
    cu = c["cu"].tolist()
    assert not bool(torch.isfinite(y[:, 100:300]).any())
    assert not bool(torch.isfinite(S_T[0]).any())
    clean = dict(c, x=c["x"].clone())
    clean["x"][:, 100] = 1.0
    ref = reference(clean, "leaky")
    for n in range(1, len(lens)):
        at = (slice(None), slice(cu[n], cu[n + 1]))
        check("sequence %d" % n, y[at], (ref["y"][0][at], ref["y"][1][at]), F32)
    check("states", S_T[1:], (ref["S_T"][0][1:], ref["S_T"][1][1:]), F32)


@pytest.mark.parametrize("scale", ["one", "leaky", "norm"])
def test_decay_at_its_ends(scale):
    """alpha = 1 (log decay 0) and alpha = 0 (-inf) among ordinary ones, and long runs of either."""
    c = make(1, 2, 700, 24, F32, s0=True, seed=6)
    c["la"][..., 3::7, :] = 0.0
    c["la"][..., 5::11, :] = float("-inf")
    c["la"][:, 0, 100:400] = 0.0
    c["la"][:, 1, 100:400] = float("-inf")
    y, S_T, entry = run_fwd(c, scale, F32)
    ref = reference(c, scale, c["dy"], c["dS_T"])
    check("y", y, ref["y"], F32)
    check("S_T", S_T, ref["S_T"], F32)
    grads = kda.glr_bwd(c["x"], c["la"], c["S0"], c["dy"], c["dS_T"], entry_states=entry, **kw(c, scale))
    for k, g in zip(("dx", "dd", "du", "dS0"), grads):
        if g is not None:
            check(k, g, ref[k], F32)


def test_slow_decay_over_many_chunks():
    """Decays so near 1 that a state lives through every chunk."""
    c = make(1, 2, 3000, 64, F32, s0=True, seed=7, la_range=(-2e-4, 0.0))
    y, S_T, entry = run_fwd(c, "one", F32)
    ref = reference(c, "one", c["dy"], c["dS_T"])
    check("y", y, ref["y"], F32)
    check("S_T", S_T, ref["S_T"], F32)
    grads = kda.glr_bwd(c["x"], c["la"], c["S0"], c["dy"], c["dS_T"], entry_states=entry, **kw(c, "one"))
    for k, g in zip(("dx", "dd", "du", "dS0"), grads):
        if g is not None:
            check(k, g, ref[k], F32)


def test_split_and_resume():
    """Prefill of a prefix, then of the rest from its state, then tokens one by one."""
    c = make(2, 2, 603, 128, BF16, z=True, u=True, s0=True, seed=8)
    ref = reference(c, "norm")
    cut = lambda t, a, b: None if t is None else t[:, :, a:b].contiguous()
    S = c["S0"].clone()
    for a, b in ((0, 256), (256, 600)):
        y, S, _ = kda.glr_fwd(cut(c["x"], a, b), None, S, S_T=S, z=cut(c["z"], a, b), A_log=c["A"], g_min=G_MIN,
                              in_gate=cut(c["u"], a, b), input_scale="norm")
        check("rows %d..%d" % (a, b), y, (ref["y"][0][:, :, a:b], ref["y"][1][:, :, a:b]), BF16)
    for t in range(600, 603):
        one = lambda k: c[k][:, :, t].contiguous()
        y = kda.glr_step(one("x"), None, S, z=one("z"), A_log=c["A"], g_min=G_MIN, in_gate=one("u"), input_scale="norm")
        check("token %d" % t, y, (ref["y"][0][:, :, t], ref["y"][1][:, :, t]), BF16)
    check("S_T", S, ref["S_T"], F32)


@pytest.mark.parametrize("packed", [False, True])
def test_no_rows(packed):
    """T = 0: the states pass through, every gradient sum is zero."""
    N, H, d = 3, 2, 10
    lead = (H, 0) if packed else (N, H, 0)
    x = torch.empty(*lead, d, device=DEV)
    cu = torch.zeros(N + 1, dtype=torch.int32, device=DEV) if packed else None
    S0, A = torch.randn(N, H, d, device=DEV), torch.zeros(H, d, device=DEV)
    y, S_T, entry = kda.glr_fwd(x, None, S0, z=x, A_log=A, in_gate=x, cu_seqlens=cu, store_entry_states=True)
    assert y.shape == x.shape and torch.equal(S_T, S0) and entry.numel() == 0
    assert not bool(kda.glr_fwd(x, x, None, cu_seqlens=cu)[1].any())
    S = S0.clone()
    assert kda.glr_fwd(x, x, S, S_T=S, cu_seqlens=cu)[1] is S and torch.equal(S, S0)
    out = kda.glr_bwd(x, None, S0, y, S0, z=x, A_log=A, in_gate=x, cu_seqlens=cu)
    assert torch.equal(out[3], S0) and not bool(out[4].any())
    assert not bool(kda.glr_bwd(x, x, S0, y, None, cu_seqlens=cu)[3].any())


def test_narrow_heads_share_tiles_and_nothing_else():
    """Heads side by side in a tile: bad numbers in one change no bit of the others, and rows behind
    the last sequence stay as they were."""
    c = make(60, 20, 300, 12, BF16, z=True, u=True, s0=True, seed=15)
    run = lambda x, dy: run_fwd(dict(c, x=x), "norm", F32)[:2] + kda.glr_bwd(
        x, None, c["S0"], dy, c["dS_T"], **kw(c, "norm"))[:4]
    clean = run(c["x"], c["dy"])
    x, dy = c["x"].clone(), c["dy"].clone()
    x[5, 7, 100], dy[31, 0, 200] = float("inf"), float("nan")
    bad = run(x, dy)
    keep = torch.ones(60, 20, dtype=torch.bool, device=DEV)
    keep[5, 7] = keep[31, 0] = False
    for want, got in zip(clean, bad):
        assert torch.equal(want[keep], got[keep])
    assert not bool(torch.isfinite(bad[0][5, 7, 100:]).any()) and not bool(torch.isfinite(bad[2][31, 0, :201]).any())

    p = make(0, 700, 0, 7, F32, lens=[70, 200], z=True, u=True, s0=True, tail=40, seed=16)
    y, S_T, entry = run_fwd(p, "leaky", F32)
    for k in ("x", "z", "u", "dy"):
        p[k][:, 270:] = float("nan")
    y2, S2, _ = run_fwd(p, "leaky", F32)
    assert bool((y2[:, 270:] == GUARD).all()) and torch.equal(y2, y) and torch.equal(S2, S_T)
    for g in kda.glr_bwd(p["x"], None, p["S0"], p["dy"], p["dS_T"], entry_states=entry, **kw(p, "leaky")):
        assert bool(torch.isfinite(g[:, :270] if g.dim() == 3 and g.shape[1] == 310 else g).all())


def test_bad_gradients_stay_in_their_sequence():
    lens = [300, 5, 256, 0, 190, 1]
    c = make(0, 2, 0, 64, F32, lens=lens, u=True, s0=True, seed=14)
    dy = c["dy"].clone()
    dy[:, 400] = float("nan")                        # sequence 2, rows 305..560
    dx, dd, du, dS0, _ = kda.glr_bwd(c["x"], c["la"], c["S0"], dy, c["dS_T"], **kw(c, "leaky"))
    ref = reference(c, "leaky", c["dy"], c["dS_T"])
    cu = c["cu"].tolist()
    for n in (0, 1, 4, 5):
        at = (slice(None), slice(cu[n], cu[n + 1]))
        for k, g in (("dx", dx), ("dd", dd), ("du", du)):
            check("%s of sequence %d" % (k, n), g[at], (ref[k][0][at], ref[k][1][at]), F32)
        check("dS0 of sequence %d" % n, dS0[n], (ref["dS0"][0][n], ref["dS0"][1][n]), F32)
    after = (slice(None), slice(401, cu[3]))         # behind the bad row of its own sequence: untouched
    check("dx behind it", dx[after], (ref["dx"][0][after], ref["dx"][1][after]), F32)
    assert not bool(torch.isfinite(dx[:, cu[2]:401]).any()) and not bool(torch.isfinite(dS0[2]).any())


@pytest.mark.parametrize("fill", [0, 0x5a, 0xff])
def test_one_workspace_for_many_calls(fill):
    """A caller's workspace, whatever it holds, serves calls of any shape one after the other."""
    ws = torch.full((64 << 20,), fill, dtype=torch.uint8, device=DEV)
    for i, (N, H, T, d, lens) in enumerate([(2, 3, 900, 72, None), (0, 2, 0, 130, [400, 0, 3, 700]), (1, 1, 1500, 33, None)]):
        c = make(N, H, T, d, BF16, lens=lens, z=True, u=True, s0=True, seed=30 + i)
        k = kw(c, "norm")
        dy = c["dy"].to(BF16)
        want = kda.glr_fwd(c["x"], None, c["S0"], **k)[:2] + kda.glr_bwd(c["x"], None, c["S0"], dy, c["dS_T"], **k)
        got = (kda.glr_fwd(c["x"], None, c["S0"], workspace=ws, **k)[:2]
               + kda.glr_bwd(c["x"], None, c["S0"], dy, c["dS_T"], workspace=ws, **k))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits():
    """2.2e9 elements (T x d past 2^31): the last rows against the same rows run alone from the state
    that the long call had there."""
    T, d = (1 << 31) // 1024 + 70000, 1024
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(1, 1, 4096, d, generator=g, device=DEV).to(BF16).repeat(1, 1, -(-T // 4096), 1)[:, :, :T].contiguous()
    la = (torch.rand(1, 1, 4096, d, generator=g, device=DEV) * -0.5).to(BF16).repeat(1, 1, -(-T // 4096), 1)[:, :, :T].contiguous()
    y, S_T, entry = kda.glr_fwd(x, la, None, store_entry_states=True)
    at = (T // kda.GLR_CHUNK - 3) * kda.GLR_CHUNK
    cut = lambda t: t[:, :, at:].contiguous()
    y2, S2, _ = kda.glr_fwd(cut(x), cut(la), entry[:, at // kda.GLR_CHUNK].reshape(1, 1, d).contiguous())
    torch.cuda.synchronize()
    # the same recurrence from the same state; tiles that start elsewhere may round differently
    assert bool(((y[:, :, at:].float() - y2.float()).abs() <= 2.0 ** -7 * y2.float().abs() + 1e-5).all())
    assert bool(((S_T - S2).abs() <= 2.0 ** -16 * S2.abs() + 1e-5).all())
    # and the head of it against the token loop
    n = 300
    q = glr.gates(host32(x[0, 0, :n]), host32(la[0, 0, :n]))
    hs, _, _ = glr.forward(q, np.zeros(d))
    hb, _ = glr.forward_bound(q, np.zeros(d), "one")
    check("head", y[0, 0, :n], (hs, hb), BF16)


def test_same_bits_every_call():
    c = make(0, 4, 0, 128, BF16, lens=[1500, 20, 3000, 700], z=True, u=True, s0=True, seed=9)
    first = None
    for _ in range(5):
        y, S_T, entry = run_fwd(c, "norm", BF16)
        grads = kda.glr_bwd(c["x"], None, c["S0"], c["dy"].to(BF16), c["dS_T"], entry_states=entry, **kw(c, "norm"))
        out = [y, S_T] + list(grads)
        if first is None:
            first = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_captured_replay_and_side_stream():
    """One workspace and one graph: replays with new inputs copied in give the eager results; the
    eager call on another stream gives them too."""
    c = make(1, 4, 1500, 128, BF16, z=True, u=True, s0=True, seed=10)
    c2 = make(1, 4, 1500, 128, BF16, z=True, u=True, s0=True, seed=11)
    y, S_T = torch.empty_like(c["x"]), torch.empty_like(c["S0"])
    k = kw(c, "norm")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kda.glr_fwd(c["x"], None, c["S0"], y=y, S_T=S_T, stream=side, **k)
    side.synchronize()
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.glr_fwd(c["x"], None, c["S0"], y=y, S_T=S_T, **k)
        grads = kda.glr_bwd(c["x"], None, c["S0"], y, S_T, **k)
    eager = None
    for i in range(4):
        if i == 2:
            for n in ("x", "z", "u", "S0"):
                c[n].copy_(c2[n])
        y.fill_(GUARD)
        graph.replay()
        torch.cuda.synchronize()
        got = [y.clone(), S_T.clone()] + [t.clone() for t in grads]
        ye, Se, _ = kda.glr_fwd(c["x"], None, c["S0"], **k)
        eager = [ye, Se] + list(kda.glr_bwd(c["x"], None, c["S0"], ye, Se, **k))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager))
        if i < 2:
            assert torch.equal(got[0], want)


def test_two_streams_at_once():
    cs = [make(1, 8, 4000, 128, BF16, z=True, u=True, s0=True, seed=20 + i) for i in range(2)]
    want = [kda.glr_fwd(c["x"], None, c["S0"], **kw(c, "norm"))[:2] for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for _ in range(8):
        for i, c in enumerate(cs):
            got[i] = kda.glr_fwd(c["x"], None, c["S0"], stream=streams[i], **kw(c, "norm"))[:2]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
