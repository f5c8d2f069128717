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
