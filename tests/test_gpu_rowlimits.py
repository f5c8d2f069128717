"""The vocabulary operators at the limits of their kernels: sizes where a
kernel's view of a row and the host's differ, wide gaps between listed and
unlisted tokens, rows that hold a NaN, and long batches."""
import numpy as np
import pytest
import torch

import rowloss_ref as ref
import sparse_gradient_synchronization_amd as sg
from gpu_util import need_gpu
from test_gpu_rowloss import TDT, check, dev, host, make_logits

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# top logits
# ---------------------------------------------------------------------------
# One line of 8 chunks more than the LDS holds, where an unaligned row or the
# last part of a split row has a chunk or more less: V / VEC = 65537 and its
# neighbours; the whole row, and parts of 8194 lines whose last has 8186.
@pytest.mark.parametrize("T,V,k,dtype,ld,shift", [
    (130, 262147, 64, "f32", None, 1), (130, 262148, 64, "f32", None, 3), (130, 262149, 64, "f32", None, 0),
    (130, 262150, 300, "f32", 262157, 2), (130, 262152, 5, "f32", None, 1), (130, 262176, 64, "f32", None, 1),
    (129, 524295, 64, "bf16", None, 5), (129, 524297, 64, "bf16", None, 0), (129, 524302, 256, "bf16", None, 7),
    (2, 1048577, 1024, "f32", None, 0), (2, 2097153, 1024, "bf16", None, 1), (1, 1049000, 1000, "f32", None, 1)])
def test_top_rows_around_the_most_lines(T, V, k, dtype, ld, shift):
    need_gpu()
    ld = ld or V
    g = torch.Generator(device="cuda").manual_seed(V + shift)
    buf = torch.full((T * ld + shift,), 100.0, dtype=TDT[dtype], device="cuda")
    x = buf[shift:].view(T, ld)[:, :V]
    x.copy_(torch.randn((T, V), device="cuda", generator=g) * 2)
    idx, logp, lse = sg.sg_topk_rows(x, k)
    for a in range(0, T, 16):
        rows = x[a:a + 16].double()
        first = torch.sort(rows, dim=1, descending=True, stable=True).indices[:, :k].sort(1).values
        assert torch.equal(idx[a:a + 16].long(), first), a
        want = torch.logsumexp(rows, 1)
        check(host(lse[a:a + 16]), host(want), ref.sum_error(V) + 2.0 ** -24 * np.abs(host(want)), "lse")
        z = host(rows.gather(1, first) - want[:, None])
        check(host(logp[a:a + 16]), z, ref.sum_error(V) + 2.0 ** -24 * np.abs(z), "logp")
    assert sg.sg_device_error() == 0
