"""Host-side checks of layouts that include/kda_attn.h allows or refuses (no GPU): the calls pass or fail validation,
and a call that passes it answers KDA_ERR_HIP for want of a device."""
import pytest
import torch

from gated_delta_rule_78_amd.attn import PageStrides
from tests.test_abi_attn import INVALID, UNSUPPORTED, adesc, app, att, lib, p, tdesc  # noqa: F401  (lib is the fixture)

# with a device a call that passes validation would launch on addresses that are none
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on addresses that are none")


@no_device
@pytest.mark.parametrize("stride, ok", [(0, True), (4, True), (9, True), (3, False), (1, False), (-1, False), (-4, False)])
def test_tables_of_one_row_for_every_sequence(lib, stride, ok):  # noqa: F811
    assert (att(lib, tdesc(stride=stride)) != INVALID) == ok
    assert (app(lib, adesc(stride=stride)) != INVALID) == ok


@no_device
@pytest.mark.parametrize("pages, ok", [(1, True), (2, False)])
def test_strides_between_pages_that_there_are(lib, pages, ok):  # noqa: F811
    far = PageStrides(1 << 32, 1024, 64)
    assert (att(lib, tdesc(pg=pages, kc=far, vc=far), kc=p(10), vc=p(20)) not in (INVALID, UNSUPPORTED)) == ok
