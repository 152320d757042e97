"""Pins of oracle.attn (fp64): closed forms, invariants of the rotation, central differences, and the
attention against a definition of its own."""
import numpy as np
import pytest

from oracle import attn


def test_pairs_and_quarter_turns():
    x = np.arange(1.0, 9.0)
    th = np.array([[np.pi / 2, 0.0]])                                 # the first pair a quarter turn, the second none
    half = attn.rotate(x[None], th, 4, False, 1.0)[0]
    assert np.allclose(half, [-3, 2, 1, 4, 5, 6, 7, 8], atol=1e-15)   # pairs (0, 2), (1, 3); channels 4 .. 7 stay
    inter = attn.rotate(x[None], th, 4, True, 1.0)[0]
    assert np.allclose(inter, [-2, 1, 3, 4, 5, 6, 7, 8], atol=1e-15)  # pairs (0, 1), (2, 3)
    assert np.allclose(attn.rotate(x[None], th, 4, True, 2.0)[0], [-4, 2, 6, 8, 5, 6, 7, 8], atol=1e-15)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_depends_on_the_distance_alone(inter):
    r = np.random.default_rng(1)
    q, k, f = r.standard_normal(8), r.standard_normal(8), np.array([1.0, 0.3, 0.01, 0.002], np.float32)
    dot = lambda m, n: float(attn.rotate(q, attn.angles(m, f), 8, inter, 1.0) @ attn.rotate(k, attn.angles(n, f), 8, inter, 1.0))
    assert abs(dot(7, 3) - dot(1004, 1000)) < 1e-12
    assert abs(np.linalg.norm(attn.rotate(q, attn.angles(5, f), 8, inter, 1.0)) - np.linalg.norm(q)) < 1e-14


def test_norm_by_hand():
    r = attn.head_rope(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), None, rot=0, interleaved=False, scale=1.0, norm=True, eps=0.0)
    assert np.allclose(r["z"], [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], atol=1e-15)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_gradients_against_differences(inter, norm):
    r = np.random.default_rng(2)
    x, w, dz = r.standard_normal((3, 2, 10)), 1.0 + 0.1 * r.standard_normal(10), r.standard_normal((3, 2, 10))
    th = attn.angles(np.array([0, 5, 77]), np.array([1.0, 0.1, 0.01], np.float32))[:, None]
    kw = dict(rot=6, interleaved=inter, scale=1.3, norm=norm, eps=1e-3)
    f = lambda a, b: float((attn.head_rope(a, b if norm else None, th, **kw)["z"] * dz).sum())
    g = attn.head_rope(x, w if norm else None, th, dz=dz, **kw)
    h = 1e-6
    for idx in np.ndindex(*x.shape):
        up, dn = x.copy(), x.copy()
        up[idx] += h
        dn[idx] -= h
        assert abs((f(up, w) - f(dn, w)) / (2 * h) - g["dx"][idx]) < 1e-7, idx
    for j in range(10 if norm else 0):
        up, dn = w.copy(), w.copy()
        up[j] += h
        dn[j] -= h
        assert abs((f(x, up) - f(x, dn)) / (2 * h) - g["dw"][j]) < 1e-7, j


def test_places():
    got = attn.places([1, 3, 3, 6], [4, 0, 2], [[5, 9], [0, 0], [7, 99]], 2, 10)
    assert got == [(-1, 0, -1, 0), (0, 2, 9, 0), (0, 3, 9, 1), (2, -1, -1, 1), (2, 0, 7, 0), (2, 1, 7, 1)]


def attention_by_definition(q, K, V, pos, window, scale):
    """One query over [0, pos], plainly."""
    js = [j for j in range(len(K)) if j <= pos and (window == 0 or j > pos - window)]
    if not js:
        return np.zeros(V.shape[1]), -np.inf
    e = [np.exp(scale * sum(a * b for a, b in zip(q, K[j]))) for j in js]
    return sum(x * V[j] for x, j in zip(e, js)) / sum(e), np.log(sum(e))


@pytest.mark.parametrize("window", [0, 1, 3])
def test_paged_attention_is_the_definition(window):
    r = np.random.default_rng(3)
    page, Hk, G, dk, dv, pages = 2, 2, 2, 4, 3, 9
    kc, vc = r.standard_normal((pages, Hk, page, dk)), r.standard_normal((pages, Hk, page, dv))
    table, kv, cu = [[3, 1, 4], [8, 0, 0], [2, 6, 5]], [5, 0, 2], [0, 2, 2, 6]     # the last: 4 tokens, 2 positions
    q = r.standard_normal((6, Hk * G, dk))
    o, _, lse, _ = attn.paged_attn(q, kc, vc, table, kv, cu, scale=0.7, window=window)
    for s in range(3):
        K = np.concatenate([kc[p] for p in table[s]], 1)[:, :kv[s]] if kv[s] else np.zeros((Hk, 0, dk))
        V = np.concatenate([vc[p] for p in table[s]], 1)[:, :kv[s]] if kv[s] else np.zeros((Hk, 0, dv))
        n = cu[s + 1] - cu[s]
        for i in range(n):
            for h in range(Hk * G):
                want, wl = attention_by_definition(q[cu[s] + i, h], K[h // G], V[h // G], kv[s] - n + i, window, 0.7)
                assert np.allclose(o[cu[s] + i, h], want, atol=1e-13)
                assert lse[cu[s] + i, h] == wl or abs(lse[cu[s] + i, h] - wl) < 1e-13
    assert np.isneginf(lse[2]).all() and np.isneginf(lse[3]).all() and not np.isneginf(lse[4:]).any()


@pytest.mark.parametrize("slip", ["pairs", "sign", "scale", "eps", "window", "heads", "causal"])
def test_planted_slips_fail(slip):
    """Each pin above has something to find: the slip changes a checked number."""
    r = np.random.default_rng(4)
    x, f = r.standard_normal(8), np.array([1.0, 0.3, 0.01, 0.002], np.float32)
    th = attn.angles(5, f)
    if slip in ("pairs", "sign", "scale"):
        right = attn.rotate(x, th, 8, False, 1.3)
        wrong = {"pairs": attn.rotate(x, th, 8, True, 1.3), "sign": attn.rotate(x, th, 8, False, 1.3, -1.0),
                 "scale": attn.rotate(x, th, 8, False, 1.0)}[slip]
        assert np.abs(right - wrong).max() > 1e-3
    elif slip == "eps":
        kw = dict(rot=0, interleaved=False, scale=1.0, norm=True)
        assert np.abs(attn.head_rope(x, None, None, eps=1e-1, **kw)["z"] - attn.head_rope(x, None, None, eps=0.0, **kw)["z"]).max() > 1e-3
    else:
        q, K, V = r.standard_normal(4), r.standard_normal((6, 4)), r.standard_normal((6, 3))
        base = attention_by_definition(q, K, V, 3, 2, 1.0)[0]
        wrong = {"window": attention_by_definition(q, K, V, 3, 3, 1.0)[0], "causal": attention_by_definition(q, K, V, 4, 2, 1.0)[0],
                 "heads": attention_by_definition(q, K[::-1], V, 3, 2, 1.0)[0]}[slip]
        assert np.abs(base - wrong).max() > 1e-3
