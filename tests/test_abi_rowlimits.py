"""The vocabulary operators' host checks at the limits of their arguments."""
import pytest
import torch

import sparse_gradient_synchronization_amd as sg
from test_abi_rows import SG_EINVAL, SG_OK, calls


@pytest.mark.parametrize("op", ["topk", "distill", "policy"])
def test_temperatures_whose_scale_fp32_cannot_hold(op):
    f = calls(sg.lib())[op]
    for it in (9e-38, 1e-39, 1e-45, 1e-300):
        assert f(it=it) == SG_EINVAL, it
    for it in (1e-37, 1e-30, 1e6):
        assert f(it=it, T=0) == SG_OK, it


def test_binding_refuses_a_workspace_elsewhere():
    """A large enough workspace of another device, or one whose elements lie apart, is not written to."""
    gpu = torch.device("cuda", 0)
    with pytest.raises(ValueError):
        sg._scratch(100, torch.zeros(200, dtype=torch.uint8), gpu)
    cpu = torch.device("cpu")
    with pytest.raises(ValueError):
        sg._scratch(100, torch.zeros(400, dtype=torch.uint8)[::2], cpu)
    ws = torch.zeros(50, dtype=torch.float32)
    assert sg._scratch(200, ws, cpu) == (ws, ws.data_ptr(), 200)
    assert sg._scratch(0, torch.zeros(2), gpu) == (None, None, 0)
