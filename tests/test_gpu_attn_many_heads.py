"""The attention over a paged cache with many query heads a key head: waves whose rows all belong to one
token, tokens over several waves or tiles, and what later tokens hold in the same blocks of keys."""
import numpy as np
import pytest
import torch

from tests.test_gpu_paged_attn import call, check, ids, make, tokens

pytestmark = pytest.mark.gpu

CASES = [
    # new tokens, past, Hq, Hk, dk, dv, page, window, packed
    ([10], [0], 64, 2, 64, 64, 16, 0, False),             # a wave a token
    ([10], [70], 64, 2, 128, 128, 64, 0, False),
    ([9], [30], 32, 1, 64, 128, 16, 20, False),
    ([11, 1, 5], [5, 90, 300], 48, 1, 128, 64, 16, 0, True),      # waves across two tokens
    ([20], [100], 96, 2, 128, 128, 32, 33, False),
    ([6], [40], 256, 1, 64, 64, 16, 0, False),            # a tile a token
    ([5, 3], [0, 130], 320, 1, 128, 128, 64, 0, True),    # tokens over two tiles
    ([4], [20], 512, 1, 64, 64, 48, 9, False),            # a token two tiles
    ([3], [3000], 512, 1, 128, 128, 64, 0, False),
]


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_parity(c):
    x = make(c)
    o, lse = call(c, x)
    torch.cuda.synchronize()
    check(c, x, o, lse)


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("c", CASES, ids=ids)
def test_later_tokens_reach_no_earlier_one(c, value, where):
    """A non-finite key or value of one position, the last ones among them: rows that do not see it keep their
    bits."""
    x = make(c)
    clean, clean_l = call(c, x)
    s = int(np.argmax(c[0]))
    n, kv = c[0][s], c[0][s] + c[1][s]
    for j in (kv - 1, kv - n // 2 - 1, max(0, kv - n - 5)):
        t = x["kc" if where == "k" else "vc"].clone()
        t[int(x["table"][s, j // c[6]]), :, j % c[6], 3] = value
        o, lse = call(c, dict(x, **{"kc" if where == "k" else "vc": t}))
        a, b, la, lb = (torch.from_numpy(tokens(u, c[8])) for u in (clean, o, clean_l, lse))
        sees = torch.zeros(a.shape[0], dtype=torch.bool)
        for i in range(n):
            pos = kv - n + i
            sees[x["cu_host"][s] + i] = j <= pos and (c[7] == 0 or j > pos - c[7])
        assert torch.equal(a[~sees], b[~sees]) and torch.equal(la[~sees], lb[~sees]), j
        if where == "v":
            assert not torch.isfinite(b[sees][..., 3]).any() and torch.equal(la, lb), j
            assert torch.isfinite(b[..., :3]).all() and torch.isfinite(b[..., 4:]).all(), j
