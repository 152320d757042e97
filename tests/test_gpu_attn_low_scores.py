"""The attention over a paged cache where keys that a token sees give scores of -inf."""
import numpy as np
import pytest
import torch

from tests.test_gpu_attn_nonfinite import CASES, INF, position, seen_by
from tests.test_gpu_paged_attn import call, ids, make, tokens

pytestmark = pytest.mark.gpu


def all_low(x, c, keep=()):
    """Every key of every sequence gives a score of -inf, but for the positions in `keep` of each."""
    kc, q = x["kc"].clone(), x["q"].clone()
    q[..., 3] = 1.0
    for s in range(len(c[0])):
        for j in range(c[0][s] + c[1][s]):
            if j not in keep:
                p, r = position(x, c, s, j)
                kc[p, :, r, 3] = -INF
    return dict(x, kc=kc, q=q)


@pytest.mark.parametrize("c", CASES[:4] + CASES[4:6] + CASES[7:], ids=ids)
def test_rows_whose_scores_are_all_low(c):
    """Scores of -inf throughout: lse = log 0 = -inf and o = 0 / 0 = NaN; a token that sees no position stays at 0."""
    x = all_low(make(c), c)
    kv = x["kv_lens"].clone()
    kv[0] = max(0, c[0][0] - 2)                       # the first two tokens of sequence 0 see nothing
    for lens, none in ((x["kv_lens"], 0), (kv, min(2, c[0][0]))):
        o, lse = (torch.from_numpy(tokens(t, c[8])) for t in call(c, dict(x, kv_lens=lens)))
        assert torch.isneginf(lse).all()
        assert not o[:none].any() and torch.isnan(o[none:]).all()


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_low_scores_beside_others(c):
    """A score of -inf is a probability of 0: the other keys alone make the result; times a NaN it is one, and so
    is the output."""
    if max(c[1]) > 10000:
        c = (c[0], [1200]) + c[2:]
    s = int(np.argmax(c[0]))
    n, kv = c[0][s], c[0][s] + c[1][s]
    keep = (kv - n, 0) if c[7] == 0 else tuple(range(0, kv, max(1, c[7] // 2)))
    x = all_low(make(c, fill=0.0), c, keep)
    o, lse = call(c, x)
    a, la = (torch.from_numpy(tokens(t, c[8])) for t in (o, lse))
    T = a.shape[0]
    # the same over the kept keys alone, in 64 bits
    for i in range(n):
        t, pos = x["cu_host"][s] + i, kv - n + i
        js = [j for j in keep if j <= pos and (c[7] == 0 or j > pos - c[7])]
        if not js:
            continue
        at = [position(x, c, s, j) for j in sorted(set(js))]
        K = torch.stack([x["kc"][p, :, r] for p, r in at], 1).double().cpu()       # [Hk, keys, dk]
        V = torch.stack([x["vc"][p, :, r] for p, r in at], 1).double().cpu()
        q = torch.from_numpy(tokens(x["q"], c[8])[t]).double().view(c[3], -1, c[4])
        sc = q @ K.transpose(1, 2) * float(np.float32(c[4] ** -0.5))
        P = torch.softmax(sc, -1)
        want, mag = (P @ V).reshape(c[2], c[5]), (P @ V.abs()).reshape(c[2], c[5])
        # probabilities in bf16 (2^-8), the result rounded once (2^-8); dk + 8 roundings of a score, twice in a
        # probability's quotient
        e = 2.0 ** -24 * (c[4] + 8) * float((q.abs() @ K.abs().transpose(1, 2)).max()) * c[4] ** -0.5
        tol = 2.0 ** -8 * 1.01 * (mag + want.abs()) + 2.0 * e * mag
        assert bool(((a[t].double() - want).abs() <= tol).all()), i
    # a NaN among the values of a key whose probability is 0
    j = kv - n - 1 if kv > n and kv - n - 1 not in keep else kv - 1
    if j in keep:
        return
    v = x["vc"].clone()
    p, r = position(x, c, s, j)
    v[p, :, r, 3] = float("nan")
    b, lb = (torch.from_numpy(tokens(t, c[8])) for t in call(c, dict(x, vc=v)))
    sees = seen_by(x, c, s, j)
    assert torch.isnan(b[sees][..., 3]).all()
    assert torch.equal(b[~sees].nan_to_num(7.0), a[~sees].nan_to_num(7.0)) and torch.equal(lb, la)


@pytest.mark.parametrize("c", [([1], [40], 4, 2, 128, 128, 16, 0, False), ([4, 2], [300, 120], 4, 1, 64, 64, 16, 0, True),
                               ([3], [6000], 2, 1, 64, 128, 16, 0, False), ([90], [100], 8, 2, 64, 128, 32, 0, False)], ids=ids)
def test_a_nan_value_where_a_whole_wave_has_low_scores(c):
    """The key of a NaN value and all those near it have scores of -inf: 0 times NaN all the same."""
    s = int(np.argmax(c[1]))
    n, kv = c[0][s], c[0][s] + c[1][s]
    x = all_low(make(c), c, keep=(kv - n,))
    clean, lse = (torch.from_numpy(tokens(t, c[8])) for t in call(c, x))
    own = seen_by(x, c, s, 5)
    assert torch.isfinite(clean[own]).all()
    v = x["vc"].clone()
    p, r = position(x, c, s, 5)
    v[p, :, r, 3] = float("nan")
    o, l2 = (torch.from_numpy(tokens(t, c[8])) for t in call(c, dict(x, vc=v)))
    assert torch.isnan(o[own][..., 3]).all() and torch.equal(o[own][..., 4:], clean[own][..., 4:]) and torch.equal(l2, lse)
