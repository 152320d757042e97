"""Host-side checks of layouts that include/kda_attn.h allows or refuses (no GPU): the calls pass or fail validation,
and a call that passes it answers KDA_ERR_HIP for want of a device."""
import pytest
import torch

from tests.test_abi_attn import INVALID, adesc, app, att, lib, tdesc  # noqa: F401  (lib is the fixture)

# with a device a call that passes validation would launch on addresses that are none
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on addresses that are none")


@no_device
@pytest.mark.parametrize("stride, ok", [(0, True), (4, True), (9, True), (3, False), (1, False), (-1, False), (-4, False)])
def test_tables_of_one_row_for_every_sequence(lib, stride, ok):  # noqa: F811
    assert (att(lib, tdesc(stride=stride)) != INVALID) == ok
    assert (app(lib, adesc(stride=stride)) != INVALID) == ok
