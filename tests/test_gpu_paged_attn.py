"""GPU parity of the attention over a paged cache (kda_paged_attn) with fp64. Every output element is
held to the bound that oracle.attn derives, plus half a step of bf16."""
import numpy as np
import pytest
import torch

import gated_delta_rule_78_amd as kda
from oracle import attn as ref
from tests.parity import host32, say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
BF16, F32 = torch.bfloat16, torch.float32
U16 = 2.0 ** -8

CASES = [
    # new tokens, past, Hq, Hk, dk, dv, page, window, packed
    ([1], [0], 1, 1, 64, 64, 16, 0, False),
    ([1], [299], 4, 1, 128, 128, 16, 0, False),
    ([1, 1, 1, 1], [0, 15, 16, 63], 8, 2, 128, 128, 16, 0, False),
    ([1] * 5, [127, 128, 511, 1000, 31], 16, 1, 64, 64, 32, 0, False),
    ([1, 1], [700, 3], 64, 2, 128, 64, 64, 0, False),
    ([4, 4, 4], [0, 60, 130], 8, 4, 64, 128, 16, 0, False),
    ([3, 0, 1, 7], [5, 9, 200, 64], 4, 2, 128, 128, 48, 0, True),
    ([70], [0], 2, 1, 64, 64, 16, 0, False),
    ([33, 1, 0, 65, 2], [31, 90, 4, 64, 700], 4, 1, 128, 128, 64, 0, True),
    ([129], [63], 3, 1, 64, 64, 32, 0, False),
    ([200], [150], 2, 2, 128, 128, 16, 0, False),
    ([40, 40], [100, 20], 7, 1, 128, 64, 80, 0, False),
    ([50, 1, 20], [100, 500, 3], 8, 2, 64, 64, 16, 37, True),
    ([1, 1, 1], [400, 64, 1], 4, 2, 128, 128, 16, 64, False),
    ([150], [0], 2, 1, 128, 128, 512, 1, False),
    ([1], [6000], 2, 1, 64, 64, 16, 0, False),
    ([1, 1], [5000, 0], 4, 2, 128, 128, 64, 0, False),
    ([20, 1, 3], [4000, 2500, 0], 8, 2, 64, 128, 32, 0, True),
    ([30, 1], [3000, 2900], 8, 1, 64, 64, 16, 1500, True),
]
ids = lambda c: "%dseq-%dtok-%dpast-%d+%dx%d+%d-page%d-w%d%s" % (len(c[0]), sum(c[0]), max(c[1]), c[2], c[3], c[4], c[5], c[6],
                                                               c[7], "-packed" if c[8] else "")


def make(c, seed=0, qs=2.0, fill=float("nan")):
    """Pages in random order; what no sequence holds, and rows behind a sequence's end, are `fill`."""
    new, past, Hq, Hk, dk, dv, page, window, packed = c
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + sum(new) + 31 * max(past))
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    N, T = len(new), sum(new)
    kv = [a + b for a, b in zip(new, past)]
    need = [-(-n // page) for n in kv]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device=DEV).tolist()
    kc = torch.full((pages, Hk, page, dk), fill, device=DEV, dtype=BF16)
    vc = torch.full((pages, Hk, page, dv), fill, device=DEV, dtype=BF16)
    width = max(need) + 1
    table = []
    for s, n in enumerate(need):
        row = [order.pop() for _ in range(n)]
        for i, p in enumerate(row):
            m = min(page, kv[s] - i * page)
            kc[p, :, :m] = rn(Hk, m, dk).to(BF16)
            vc[p, :, :m] = rn(Hk, m, dv).to(BF16)
        table.append(row + [-1] * (width - n))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = (qs * rn(T, Hq, dk)).to(BF16)
    q = q.transpose(0, 1) if packed else q.unflatten(0, (N, new[0])).transpose(1, 2)
    return dict(q=q, kc=kc, vc=vc, table=torch.tensor(table, dtype=torch.int32, device=DEV), cu_host=cu,
                kv_lens=torch.tensor(kv, dtype=torch.int32, device=DEV),
                cu=torch.tensor(cu, dtype=torch.int32, device=DEV) if packed else None)


def tokens(t, packed):
    """[T,H,...] on the host."""
    t = host32(t)
    if packed:
        return np.moveaxis(t, 1, 0)
    t = np.moveaxis(t, 2, 1)
    return t.reshape((-1,) + t.shape[2:])


def call(c, x, **kw):
    return kda.paged_attn(x["q"], x["kc"], x["vc"], x["table"], x["kv_lens"], cu_seqlens=x["cu"], window=c[7],
                          return_lse=True, **kw)


def check(c, x, o, lse, scale=None):
    scale = float(np.float32(c[4] ** -0.5 if scale is None else scale))
    want, bound, wl, bl = ref.paged_attn(tokens(x["q"], c[8]), host32(x["kc"]), host32(x["vc"]), x["table"].tolist(),
                                         x["kv_lens"].tolist(), x["cu_host"], scale=scale, window=c[7])
    got, gl = tokens(o, c[8]).astype(np.float64), tokens(lse, c[8]).astype(np.float64)
    tol = bound + U16 * (np.abs(want) + bound) + 2.0 ** -133
    assert got.shape == want.shape and np.all(np.isfinite(got))
    worst = float((np.abs(got - want) / tol).max()) if got.size else 0.0
    none = np.isneginf(wl)
    assert np.array_equal(np.isneginf(gl), none) and not np.any(got[none])
    worst_l = float((np.abs(gl - wl)[~none] / bl[~none]).max()) if (~none).any() else 0.0
    rms = float(np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-30))
    say("%s: worst error / bound: o %.3f, lse %.3f; relative 2-norm %.2e" % (ids(c), worst, worst_l, rms))
    assert worst <= 1.0 and worst_l <= 1.0


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_parity(c):
    x = make(c)
    say("paged_attn", ids(c))
    o, lse = call(c, x)
    torch.cuda.synchronize()
    check(c, x, o, lse)


BAD = [
    ([40], [30], 2, 1, 64, 64, 16, 0, False),
    ([1, 50, 9], [10, 100, 3], 4, 2, 128, 128, 64, 0, True),
    ([4, 4], [60, 200], 4, 1, 128, 64, 16, 20, False),
    ([90], [100], 8, 2, 64, 128, 32, 33, False),
]


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("c", BAD, ids=ids)
def test_bad_values_reach_only_rows_that_see_them(c, value, where):
    """A non-finite key or value of one position: rows that do not see it keep their bits, rows that do see
    a non-finite value get one."""
    x = make(c)
    clean, clean_l = call(c, x)
    s = len(c[0]) - 1 if c[8] else 0
    n, kv = c[0][s], c[0][s] + c[1][s]
    for j in (kv - 1, kv - n // 2 - 1, max(0, kv - n - 5)):
        t = (x["kc"] if where == "k" else x["vc"]).clone()
        page = int(x["table"][s, j // c[6]])
        t[page, 0, j % c[6], 3] = value
        y = dict(x, **{"kc" if where == "k" else "vc": t})
        o, lse = call(c, y)
        a, b, la, lb = (torch.from_numpy(tokens(u, c[8])) for u in (clean, o, clean_l, lse))
        T, Hq = a.shape[:2]
        sees = torch.zeros(T, Hq, dtype=torch.bool)
        for i in range(n):
            pos = kv - n + i
            if j <= pos and (c[7] == 0 or j > pos - c[7]):
                sees[x["cu_host"][s] + i, :Hq // c[3]] = True
        assert torch.equal(a[~sees], b[~sees]) and torch.equal(la[~sees], lb[~sees]), j
        if where == "v":
            assert not torch.isfinite(b[sees][:, 3]).any() and torch.equal(lb, la), j
            assert torch.isfinite(b[..., 4:]).all(), j
        elif value != value:
            assert torch.isnan(b[sees]).all() and torch.isnan(lb[sees]).all(), j
