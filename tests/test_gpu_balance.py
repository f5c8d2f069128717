"""The router's balance loss against its definition in 64 bits."""
import pytest
import torch

import sparse_gradient_synchronization_amd as sg
import step_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(T, E, k, dtype, seed=0, masked=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((T, E), device="cuda", generator=g) * 1.5 + torch.randn(E, device="cuda", generator=g)).to(DT[dtype])
    idx = torch.topk(x.float(), k, dim=1).indices.int().contiguous()
    live = torch.rand(T, device="cuda", generator=g) >= masked
    return x, idx, live


def check(out, x, idx, live, alpha, zc):
    val, err = ref.balance(x, idx, live, alpha, zc)
    loss, counts, prob, grad = out
    assert torch.equal(counts.long(), val["counts"])
    ref.close(prob, val["prob"], err["prob"], "prob")
    ref.close(loss, val["loss"], err["loss"], "loss")
    if grad is not None:
        ref.close(grad, val["grad"], err["grad"], "grad")
    assert sg.sg_device_error() == 0


# one row and one expert; every lane count and every number of chunks a lane,
# with columns that are and are not whole vectors; one block, several, all
SIZES = [(1, 1, 1), (3, 2, 2), (5, 4, 1), (64, 7, 3), (65, 8, 2), (200, 13, 4), (17, 60, 8), (1000, 63, 2), (1000, 64, 6),
         (90, 65, 5), (300, 128, 8), (300, 200, 4), (30, 255, 8), (700, 256, 8), (129, 257, 3), (140, 500, 8),
         (66, 512, 8), (40, 513, 4), (300, 1000, 8), (100, 1023, 16), (9, 1024, 1024), (20011, 16, 2), (30000, 3, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_sizes(T, E, k, dtype):
    need_gpu()
    x, idx, live = make(T, E, k, dtype, T + E)
    for zc in (0.0, 1e-2):
        check(sg.sg_balance_loss(x, idx, live=live, balance_coef=0.02, z_coef=zc), x, idx, live, 0.02, zc)
    out = sg.sg_balance_loss(x, idx, want_grad=False)
    assert out[3] is None
    check(out, x, idx, None, 0.01, 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [20, 3000])
def test_rows_that_do_not_count(T, dtype):
    need_gpu()
    x, idx, live = make(T, 48, 4, dtype, 3, masked=0.5)
    live[0] = False
    dirty = x.clone()
    dirty[~live] = float("nan")
    idx[~live] = 7
    a = sg.sg_balance_loss(dirty, idx, live=live, z_coef=1e-3)
    check(a, x, idx, live, 0.01, 1e-3)
    assert bool((a[3][~live] == 0).all())
    none = sg.sg_balance_loss(dirty, idx, live=torch.zeros_like(live), z_coef=1e-3)
    for t in none:
        assert bool((t == 0).all())
    # dropped experts, and one listed twice
    idx[1] = torch.tensor([-1, 48, 2 ** 31 - 1, -(2 ** 31)], device="cuda", dtype=torch.int32)
    idx[2] = 5
    check(sg.sg_balance_loss(x, idx, live=live), x, idx, live, 0.01, 0.0)


def test_no_rows():
    need_gpu()
    x, idx, live = make(4, 12, 2, "f32")
    loss, counts, prob, grad = sg.sg_balance_loss(x[:0], idx[:0])
    assert float(loss) == 0 and bool((counts == 0).all()) and bool((prob == 0).all()) and grad.shape == (0, 12)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [6, 2000])
def test_masked_logits_and_lowest_values(T, dtype):
    """-inf has probability 0; rows at the type's lowest value are ordinary rows."""
    need_gpu()
    x, idx, live = make(T, 20, 2, dtype, 1, masked=0.0)
    x[:, 3:9] = float("-inf")
    x[1] = torch.finfo(x.dtype).min
    x[2, 4:] = float("-inf")
    val, _ = ref.balance(x, idx, live, 0.01, 0.0)
    out = sg.sg_balance_loss(x, idx, live=live)
    p = torch.softmax(x.double(), 1)
    assert bool((out[2].double() - p.mean(0)).abs().max() <= 1e-6)
    assert bool((out[3][:, 3:9][torch.isinf(x[:, 3:9])] == 0).all()) and bool(torch.isfinite(out[3]).all())
    assert bool((out[3].double() - val["grad"]).abs().max() <= 2.0 ** -7 * val["grad"].abs().max())


@pytest.mark.parametrize("T", [6, 2000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite(T, bad):
    need_gpu()
    x, idx, live = make(T, 33, 2, "f32", 1, masked=0.0)
    ok = sg.sg_balance_loss(x, idx, live=live)
    x[4, 7] = bad
    loss, counts, prob, grad = sg.sg_balance_loss(x, idx, live=live)
    rest = torch.arange(T, device="cuda") != 4
    assert bool(loss.isnan()) and bool(prob.isnan().all()) and bool(grad[4].isnan().all())
    assert torch.equal(grad[rest], ok[3][rest]) and torch.equal(counts, ok[1])


def test_strides_and_in_place():
    need_gpu()
    for dtype in ("bf16", "f32"):
        for off, pad in [(0, 4), (1, 3), (4, 8)]:
            for E in (24, 25):
                x, idx, live = make(300, E, 3, dtype, E)
                buf = torch.full((301 * (E + pad),), 9.0, device="cuda", dtype=x.dtype)
                v = buf[off:off + 300 * (E + pad)].view(300, E + pad)[:, :E]
                v.copy_(x)
                want = sg.sg_balance_loss(x, idx, live=live)
                got = sg.sg_balance_loss(v, idx, live=live, grad=v)
                check((got[0], got[1], got[2], v.clone()), x, idx, live, 0.01, 0.0)
                rest = torch.ones_like(buf, dtype=torch.bool)
                rest[off:off + 300 * (E + pad)].view(300, E + pad)[:, :E] = False
                assert bool((buf[rest] == 9.0).all())
                assert torch.equal(got[1], want[1])


def test_same_bits_streams_and_graph():
    need_gpu()
    for T, E in ((12, 40), (5000, 64)):
        x, idx, live = make(T, E, 4, "f32")
        want = sg.sg_balance_loss(x, idx, live=live, z_coef=1e-3)
        need = sg.lib().sg_balance_workspace_bytes(T, E, 4, 0)
        ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = sg.sg_balance_loss(x, idx, live=live, z_coef=1e-3, workspace=ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        sx, si, sl = x.clone(), idx.clone(), live.clone()
        with torch.cuda.graph(graph):
            cap = sg.sg_balance_loss(sx, si, live=sl, z_coef=1e-3)
        for seed in range(4):
            nx, ni, nl = make(T, E, 4, "f32", seed, 0.1 * seed)
            sx.copy_(nx), si.copy_(ni), sl.copy_(nl)
            graph.replay()
            eager = sg.sg_balance_loss(nx, ni, live=nl, z_coef=1e-3)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(eager, cap))


def test_gradient_against_differences():
    need_gpu()
    x, idx, live = make(50, 30, 3, "f32")
    out = sg.sg_balance_loss(x, idx, live=live, balance_coef=0.5, z_coef=0.1)
    d = torch.randn(x.shape, device="cuda", dtype=torch.float64, generator=torch.Generator(device="cuda").manual_seed(2))
    f = [_loss64(x.double() + s * 1e-5 * d, idx, live) for s in (1, -1)]
    slope, terms = float(f[0] - f[1]) / 2e-5, out[3].double() * d
    assert abs(slope - float(terms.sum())) <= 1e-6 * float(terms.abs().sum()) + 1e-8


def _loss64(z, idx, live):
    n, E = float(live.sum()), z.shape[1]
    f = torch.bincount(idx[live].reshape(-1).long(), minlength=E).double() / (idx.shape[1] * n)
    q = torch.softmax(z[live], 1).sum(0) / n
    return 0.5 * E * (f * q).sum() + 0.1 * torch.logsumexp(z[live], 1).square().sum() / n
