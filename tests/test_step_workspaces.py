"""What the router's, the layer norm's and the update's calls take for a workspace (no GPU needed:
stand-ins for tensors)."""
from types import SimpleNamespace

import pytest
import torch

from activated_mlp_gemms_gb300 import router_op


def tensor(**change):
    t = dict(is_cuda=True, dtype=torch.uint8, is_contiguous=lambda: True, get_device=lambda: 0)
    return SimpleNamespace(**{**t, **change})


@pytest.mark.parametrize("change", [dict(is_cuda=False), dict(dtype=torch.int8),
                                    dict(is_contiguous=lambda: False),
                                    dict(get_device=lambda: 1)])  # another device's memory
def test_workspaces_that_are_refused(change):
    here = torch.device("cuda", 0)
    ok = tensor()
    assert router_op._ws(ok, 256, here, None) is ok
    with pytest.raises(ValueError):
        router_op._ws(tensor(**change), 256, here, None)
