"""What the elementwise bindings check of a launch's stream (no GPU)."""
from types import SimpleNamespace

import pytest
import torch

from gated_delta_rule_78_amd import _launch


@pytest.mark.parametrize("device", ["cuda:1", "cuda:3"])
def test_stream_of_another_device_is_refused(device):
    stream = SimpleNamespace(device=torch.device(device), cuda_stream=0)
    with pytest.raises(ValueError, match=r"stream is on %s, the tensors on cuda:0" % device):
        _launch.scope(0, stream)
