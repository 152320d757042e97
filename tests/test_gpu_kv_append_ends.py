"""The append to a paged cache with many tokens a workgroup: sequences that begin, end and are empty inside one,
rows that no sequence holds, and values of widths off a power of two."""
import pytest
import torch

import gated_delta_rule_78_amd as kda
from tests.test_gpu_head_rope import BF16, DEV, F32, akw, check_append, make_append

pytestmark = pytest.mark.gpu

# new tokens, past, Hq, Hk, dk, dv, rot, page, dtype, interleaved, norm, packed
RAGGED = [(s * 7) % 10 if s % 11 else 0 for s in range(2100)]


@pytest.mark.parametrize("c", [
    (RAGGED, [s % 5 for s in range(2100)], 2, 1, 64, 64, 64, 16, BF16, False, True, True),
    (RAGGED, [s % 3 for s in range(2100)], 0, 1, 32, 40, 32, 48, F32, True, True, True),
    ([3] * 3000, [s % 17 for s in range(3000)], 1, 1, 64, 24, 0, 16, BF16, False, False, False),
    ([300, 0, 50], [20, 3, 0], 2, 2, 64, 300, 64, 16, F32, False, True, True),
    ([40, 9], [0, 15], 3, 3, 128, 200, 64, 16, BF16, False, True, True),
    ([6, 6], [1, 0], 2, 1, 64, 7, 64, 16, BF16, False, True, False),
])
def test_places(c):
    x = make_append(c)
    kc, vc = x["kc"].clone(), x["vc"].clone()
    q = kda.kv_append(x["q"], x["k"], x["v"], kc, vc, x["table"], x["kv_lens"], x["f"], **akw(c, x))
    check_append(c, x, q, kc, vc, x["kc"], x["vc"])


def test_rows_before_and_behind_in_workgroups_of_many_tokens():
    c = ([0, 4000, 0, 4300, 1, 0], [3, 2, 0, 20, 5, 6], 2, 1, 64, 64, 64, 16, BF16, False, True, True)
    x = make_append(c)
    wide = lambda t: torch.cat((t[:, :5], t, t[:, :23]), 1)
    x["cu"] = x["cu"] + 5
    kc, vc = x["kc"].clone(), x["vc"].clone()
    T = 8301
    out = torch.full((2, T + 28, 64), 7.0, dtype=BF16, device=DEV)
    kda.kv_append(wide(x["q"]), wide(x["k"]), wide(x["v"]), kc, vc, x["table"], x["kv_lens"], x["f"], q_out=out, **akw(c, x))
    check_append(c, x, out[:, 5:T + 5], kc, vc, x["kc"], x["vc"])
    assert bool((out[:, :5] == 7).all()) and bool((out[:, T + 5:] == 7).all())


def test_lengths_that_break_the_rules_write_only_pages_of_the_table():
    """cu_seqlens that fall, start below 0 or end past T, kv_lens out of range: numbers are undefined, every access
    stays within the tensors, and pages that the table does not name keep their bits."""
    c = ([30, 20, 10], [3, 20, 0], 2, 1, 64, 64, 64, 16, BF16, False, True, True)
    x = make_append(c)
    spare = [p for p in range(x["pages"]) if p not in set(x["table"].flatten().tolist())]
    assert spare
    for cu, kv in (([0, 50, 30, 60], None), ([-5, 20, 40, 60], None), ([0, 30, 50, 1000], None), ([9, 9, 9, 9], None),
                   ([0, 30, 50, 60], [-7, 1 << 30, 10])):
        kc, vc = x["kc"].clone(), x["vc"].clone()
        lens = x["kv_lens"] if kv is None else torch.tensor(kv, dtype=torch.int32, device=DEV)
        kw = dict(akw(c, x), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
        kda.kv_append(x["q"], x["k"], x["v"], kc, vc, x["table"], lens, x["f"], **kw)
        assert torch.equal(kc[spare], x["kc"][spare]) and torch.equal(vc[spare], x["vc"][spare])
