"""Entry points that take a device, given its name."""
import pytest
import torch

import transformer_xl_relative_attn_gb300 as txl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("device", [0, "cuda", "cuda:0", torch.device("cuda"), torch.device("cuda", 0), None])
def test_device_names(device):
    assert txl.sync_status(device=device) == 0
    assert txl.attn_workspace_bytes(1, 2, 128, 1500, 64, device=device) == txl.attn_workspace_bytes(1, 2, 128, 1500, 64)
    assert (txl.layer_norm_bwd_workspace_bytes(20000, 500, device=device) ==
            txl.layer_norm_bwd_workspace_bytes(20000, 500) > 0)
    assert (txl.linear_bwd_workspace_bytes((1, 20000, 128), 136, device=device) ==
            txl.linear_bwd_workspace_bytes((1, 20000, 128), 136) > 0)
