"""The example: losses over a vocabulary, their gradients through the sparse
synchronization path, and an update that lowers the loss."""
import os
import sys

import pytest

from gpu_util import need_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("loss", ["distill", "policy", "preference"])
def test_head_learns(loss):
    need_gpu()
    import sparse_gradient_synchronization_amd as sg
    import train_head
    curve = train_head.train(loss, steps=12)
    # the last three steps against the first three: the batches differ from step to step
    assert sum(curve[-3:]) < 0.9 * sum(curve[:3]) if loss != "policy" else sum(curve[-3:]) < sum(curve[:3])
    assert sg.sg_device_error() == 0
