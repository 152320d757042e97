"""The attention over a paged cache where keys or values that a token sees are not finite: what the formula
gives, whichever kind of tile, block or chunk they fall in."""
import numpy as np
import pytest
import torch

from tests.test_gpu_paged_attn import call, ids, make, tokens

pytestmark = pytest.mark.gpu
INF = float("inf")

CASES = [
    # new tokens, past, Hq, Hk, dk, dv, page, window, packed
    ([1], [40], 4, 2, 128, 128, 16, 0, False),            # narrow tiles: one chunk
    ([4, 4], [60, 200], 4, 1, 128, 64, 16, 20, False),    # with a window
    ([5], [6000], 2, 1, 64, 64, 16, 0, False),            # cut
    ([40], [30], 2, 1, 64, 64, 16, 0, False),
    ([1, 50, 9], [10, 100, 3], 4, 2, 128, 128, 64, 0, True),
    ([90], [100], 8, 2, 64, 128, 32, 33, False),          # wide tiles, with a window
    ([150], [20000], 2, 1, 128, 128, 512, 0, False),      # cut
    ([10], [70], 64, 2, 128, 128, 64, 0, False),
]


def position(x, c, s, j):
    return int(x["table"][s, j // c[6]]), j % c[6]


def seen_by(x, c, s, j):
    """[T]: the tokens that see position j of sequence s."""
    n, kv = c[0][s], c[0][s] + c[1][s]
    sees = torch.zeros(x["cu_host"][-1], dtype=torch.bool)
    for i in range(n):
        pos = kv - n + i
        sees[x["cu_host"][s] + i] = j <= pos and (c[7] == 0 or j > pos - c[7])
    return sees


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_infinite_values(c):
    """sum p v with p > 0: an infinity where the values seen hold infinities of one sign, NaN where of both."""
    x = make(c)
    clean = torch.from_numpy(tokens(call(c, x)[0], c[8]))
    s = int(np.argmax(c[0]))
    n, kv = c[0][s], c[0][s] + c[1][s]
    up, down = kv - 1 - n // 2, max(kv - n - 3, 0)          # both under masks of some rows, or of the window
    for plus, minus in (((up,), ()), ((), (up,)), ((up,), (down,)), ((kv - 1,), (up,)), ((down,), ())):
        v = x["vc"].clone()
        pos, neg = torch.zeros(clean.shape[0], dtype=torch.bool), torch.zeros(clean.shape[0], dtype=torch.bool)
        for js, value, hit in ((plus, INF, pos), (minus, -INF, neg)):
            for j in js:
                p, r = position(x, c, s, j)
                v[p, :, r, 3] = value
                hit |= seen_by(x, c, s, j)
        if set(plus) & set(minus):
            continue
        o, lse = call(c, dict(x, vc=v))
        b = torch.from_numpy(tokens(o, c[8]))
        ch = b[..., 3]
        assert bool((ch[pos & ~neg] == INF).all()) and bool((ch[neg & ~pos] == -INF).all()), (plus, minus)
        assert bool(torch.isnan(ch[pos & neg]).all()), (plus, minus)
        assert torch.equal(ch[~pos & ~neg], clean[..., 3][~pos & ~neg]), (plus, minus)
        assert torch.isfinite(b[..., :3]).all() and torch.isfinite(b[..., 4:]).all()
