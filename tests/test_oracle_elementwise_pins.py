"""Pins of oracle.glr and oracle.block_norm (fp64): closed forms and central differences."""
import numpy as np
import pytest

from oracle import block_norm, glr


def case(T=9, C=4, z=False, u=False, seed=0):
    r = np.random.default_rng(seed)
    c = dict(x=r.standard_normal((T, C)), S0=r.standard_normal(C), dy=r.standard_normal((T, C)), dS=r.standard_normal(C))
    c["la"] = None if z else -r.uniform(0.001, 2.0, (T, C))
    c["z"] = r.standard_normal((T, C)) if z else None
    c["A"] = r.uniform(-0.5, 0.5, C) if z else None
    c["u"] = r.standard_normal((T, C)) if u else None
    return c


def run(c, scale):
    q = glr.gates(c["x"], c["la"], c["z"], c["A"], -5.0, c["u"], scale)
    h, prev, last = glr.forward(q, c["S0"])
    return q, h, prev, last


def test_closed_forms():
    x = np.ones((5, 1))
    h = glr.forward(glr.gates(x, la=np.full((5, 1), np.log(0.5))), np.zeros(1))[0][:, 0]
    assert np.allclose(h, [1, 1.5, 1.75, 1.875, 1.9375], atol=1e-15)
    h = glr.forward(glr.gates(x, la=np.full((5, 1), np.log(0.5)), scale="leaky"), np.ones(1))[0]
    assert np.allclose(h, 1.0, atol=1e-15)                       # a moving average of ones stays one
    h = glr.forward(glr.gates(x, la=np.zeros((5, 1)), scale="norm"), np.full(1, 3.0))[0]
    assert np.array_equal(h, np.full((5, 1), 3.0))               # alpha = 1 writes nothing
    h = glr.forward(glr.gates(x, la=np.full((5, 1), -np.inf), scale="norm"), np.full(1, 3.0))[0]
    assert np.array_equal(h, x)                                  # alpha = 0 keeps nothing
    q = glr.gates(x, z=np.zeros((5, 1)), A=np.zeros(1), u=np.zeros((5, 1)))
    assert np.allclose(q["la"], -2.5) and np.allclose(q["i"], 0.5)


def test_prefix_then_rest_is_the_whole():
    c = case()
    q, h, _, last = run(c, "norm")
    first = {k: (v[:4] if v is not None and k in ("x", "la") else v) for k, v in c.items()}
    rest = {k: (v[4:] if v is not None and k in ("x", "la") else v) for k, v in c.items()}
    mid = run(first, "norm")[3]
    assert np.allclose(run(dict(rest, S0=mid), "norm")[1], h[4:], atol=1e-14)


@pytest.mark.parametrize("scale", ["one", "leaky", "norm"])
@pytest.mark.parametrize("z,u", [(False, False), (True, True)])
def test_gradients_are_the_differences(scale, z, u):
    c = case(z=z, u=u, seed=3)
    q, h, prev, last = run(c, scale)
    g = glr.backward(q, prev, c["dy"], c["dS"])
    loss = lambda cc: (lambda r: (r[1] * c["dy"]).sum() + (r[3] * c["dS"]).sum())(run(cc, scale))
    pairs = [("x", g["dx"]), ("S0", g["dS0"]), ("z" if z else "la", g["dd"])]
    if z:
        pairs.append(("A", g["dA"]))
    if u:
        pairs.append(("u", g["du"]))
    for key, grad in pairs:
        num = np.zeros_like(c[key])
        for at in np.ndindex(*c[key].shape):
            v = []
            for s in (1e-6, -1e-6):
                m = c[key].copy()
                m[at] += s
                v.append(loss(dict(c, **{key: m})))
            num[at] = (v[0] - v[1]) / 2e-6
        assert np.allclose(num, grad, rtol=1e-6, atol=1e-8), key


@pytest.mark.parametrize("gate,res,post,pre", [(1, 1, 1, 1), (0, 1, 1, 1), (1, 0, 1, 0), (1, 1, 0, 1), (0, 1, 1, 0)])
def test_norm_gradients_are_the_differences(gate, res, post, pre):
    r = np.random.default_rng(5)
    R, D = 3, 6
    c = dict(f=r.standard_normal((R, D)), x=r.standard_normal((R, D)) if res else None,
             gate=r.standard_normal((R, D)) if gate else None, w_post=r.uniform(0.5, 1.5, D) if post else None,
             lam=r.uniform(0.5, 1.5, D), w_pre=r.uniform(0.5, 1.5, D) if pre else None)
    dxo, dn = r.standard_normal((R, D)), r.standard_normal((R, D)) if pre else None
    kw = dict(post=bool(post), pre=bool(pre), scale=0.6, eps=1e-3, pre_eps=1e-2)

    def loss(cc):
        o = block_norm.evaluate(*[cc[k] for k in ("f", "x", "gate", "w_post", "lam", "w_pre")], **kw)
        return (o["x_out"] * dxo).sum() + ((o["n"] * dn).sum() if pre else 0.0)

    o = block_norm.evaluate(*[c[k] for k in ("f", "x", "gate", "w_post", "lam", "w_pre")], dxo=dxo, dn=dn, **kw)
    for key, name in (("f", "df"), ("x", "dx"), ("gate", "dgate"), ("w_post", "dw_post"), ("lam", "dlam"), ("w_pre", "dw_pre")):
        if c[key] is None:
            continue
        num = np.zeros_like(c[key])
        for at in np.ndindex(*c[key].shape):
            v = []
            for s in (1e-6, -1e-6):
                m = c[key].copy()
                m[at] += s
                v.append(loss(dict(c, **{key: m})))
            num[at] = (v[0] - v[1]) / 2e-6
        assert np.allclose(num, o[name], rtol=1e-6, atol=1e-8), key


def test_norm_closed_form():
    """f = (3, 4): rms 5 / sqrt 2; residual 1, no gate."""
    o = block_norm.evaluate(np.array([[3.0, 4.0]]), np.ones((1, 2)), None, None, None, None, post=True, pre=True,
                            scale=2.0, eps=0.0, pre_eps=0.0)
    p = np.array([3.0, 4.0]) * np.sqrt(2.0) / 5.0
    xo = 1.0 + 2.0 * p
    assert np.allclose(o["x_out"][0], xo) and np.allclose(o["n"][0], xo / np.sqrt((xo ** 2).mean()))


def test_planted_slips_fail_the_pins():
    """A state read before its decay, and a residual scale left out of dlam, are seen."""
    c = case(seed=7)
    q, h, prev, last = run(c, "one")
    g = glr.backward(q, prev, c["dy"], c["dS"])
    wrong = glr.backward(dict(q, a=np.ones_like(q["a"])), prev, c["dy"], c["dS"])
    assert not np.allclose(g["dla"], wrong["dla"])
