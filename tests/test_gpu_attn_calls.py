"""Calls of the attention layers' operators that their documentation allows."""
import pytest
import torch

from tests.test_gpu_paged_attn import call, make

pytestmark = pytest.mark.gpu


def test_a_scale_held_in_a_tensor_is_read_at_every_call():
    c = ([1, 1], [200, 40], 4, 2, 64, 64, 16, 0, False)
    x = make(c)
    held = torch.tensor(0.125, dtype=torch.float64)
    for value in (0.125, 0.5, -0.25):
        held.fill_(value)
        o, lse = call(c, x, scale=held)
        a, al = call(c, x, scale=value)
        assert torch.equal(o, a) and torch.equal(lse, al), value
