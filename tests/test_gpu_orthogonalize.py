"""The orthogonalised update against its definition in 64 bits."""
import pytest
import torch

import sparse_gradient_synchronization_amd as sg
import step_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
MUON = (3.4445, -4.7750, 2.0315)
CUBIC = (1.5, -0.5, 0.0)


def make(shape, dtype, seed=0, scale=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m, n = shape[-2:]
    r = min(4, m, n)
    low = torch.randn(shape[:-1] + (r,), device="cuda", generator=g) @ torch.randn(shape[:-2] + (r, n), device="cuda", generator=g)
    return ((low + torch.randn(shape, device="cuda", generator=g)) * scale).to(DT[dtype])


def check(out, u, steps=5, coef=MUON, eps=1e-7):
    want, bound = ref.orthogonalize_error(u, steps, coef, eps)
    off = (out.double() - want).square().sum((-2, -1)).sqrt()
    assert out.dtype == u.dtype and out.shape == u.shape
    assert bool((off <= bound).all()), (off / bound).max()
    assert sg.sg_device_error() == 0


SIZES = [(1, 1), (1, 5), (7, 1), (3, 2), (16, 16), (33, 65), (64, 64), (65, 33), (100, 300), (127, 129), (256, 64), (130, 1000),
         (513, 200), (300, 301), (1, 2, 3), (3, 64, 100), (5, 130, 60), (2, 257, 255), (24, 40, 40)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SIZES)
def test_sizes(shape, dtype):
    need_gpu()
    u = make(shape, dtype, sum(shape))
    check(sg.sg_orthogonalize(u), u)
    check(sg.sg_orthogonalize(u, steps=1), u, 1)
    check(sg.sg_orthogonalize(u, steps=12, coef=CUBIC), u, 12, CUBIC)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1500, 4300), (4300, 1500), (20, 700, 800), (6, 1300, 600), (2100, 2100)])
def test_large_tiles(shape, dtype):
    need_gpu()
    u = make(shape, dtype, 1)
    check(sg.sg_orthogonalize(u), u)


# what the rule on tiles and parts of k chooses between: short and long k at a small side (the product in parts,
# joined; four groups of a block on one tile), many small matrices, one of some hundreds
VARIANTS = [(64, 5000), (5000, 64), (130, 3300), (3300, 130), (256, 512), (512, 256), (40, 70, 50), (9, 512, 128),
            (512, 512), (640, 2600), (2600, 640)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", VARIANTS)
def test_variants(shape, dtype):
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    u = torch.randn(shape, device="cuda", generator=g).to(DT[dtype])
    check(sg.sg_orthogonalize(u), u)
    check(sg.sg_orthogonalize(u, steps=1), u, steps=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_singular_values(dtype):
    """Known singular values: the result has the polynomial's, in the same directions."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.linalg.qr(torch.randn((96, 96), device="cuda", dtype=torch.float64, generator=g)).Q
    r = torch.linalg.qr(torch.randn((160, 96), device="cuda", dtype=torch.float64, generator=g)).Q
    s = torch.logspace(0, -2, 96, device="cuda", dtype=torch.float64)
    u = (q * s @ r.t().contiguous()).to(DT[dtype])
    t = s / (s.square().sum().sqrt() + 1e-7)
    for _ in range(5):
        t = t * (MUON[0] + t * t * (MUON[1] + t * t * MUON[2]))
    out = sg.sg_orthogonalize(u).double()
    # what the input's own rounding (half a step an element, times at most 3.5 a step) may change
    slack = 0.05 if dtype == "bf16" else 1e-4
    assert bool((torch.diagonal(q.t().contiguous() @ out @ r) - t).abs().max() < slack)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-36, 1e-20, 1.0, 1e18, 1e36])
def test_scales(scale, dtype):
    """The norm takes the scale away, also where its square is no fp32 number; eps beside a small norm."""
    need_gpu()
    u = make((60, 90), dtype, 2, 1.0)
    u = (u.float() * scale).to(u.dtype)
    check(sg.sg_orthogonalize(u, eps=0.0), u, eps=0.0)
    check(sg.sg_orthogonalize(u, eps=1e-3), u, eps=1e-3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zeros_and_not_finite(dtype):
    need_gpu()
    for shape in ((3, 70, 40), (3, 40, 70)):
        u = make(shape, dtype)
        ok = sg.sg_orthogonalize(u)
        u[1] = 0
        out = sg.sg_orthogonalize(u)
        assert bool((out[1] == 0).all()) and torch.equal(out[0], ok[0]) and torch.equal(out[2], ok[2])
        for bad in (float("nan"), float("inf"), float("-inf")):
            v = u.clone()
            v[1, 5, 7] = bad
            out = sg.sg_orthogonalize(v)
            assert bool(out[1].isnan().all()) and torch.equal(out[0], ok[0]) and torch.equal(out[2], ok[2])
    u = make((40, 40), dtype)
    u[3:] = 0  # rank 3
    check(sg.sg_orthogonalize(u), u)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_in_place_and_rest(dtype):
    need_gpu()
    for off, pad in [(0, 8), (1, 3), (4, 12), (3, 0)]:
        for B, m, n in [(1, 50, 70), (3, 41, 30)]:
            u = make((B, m, n), dtype)
            buf = torch.full((off + B * (m + 2) * (n + pad),), 5.0, device="cuda", dtype=u.dtype)
            v = buf[off:].view(B, m + 2, n + pad)[:, :m, :n]
            v.copy_(u)
            want = sg.sg_orthogonalize(u)
            rest = torch.ones_like(buf, dtype=torch.bool)
            rest[off:].view(B, m + 2, n + pad)[:, :m, :n] = False
            assert torch.equal(sg.sg_orthogonalize(v), want)
            sg.sg_orthogonalize(v, out=v)
            assert torch.equal(v, want) and bool((buf[rest] == 5.0).all())
    u = make((60, 44), dtype)
    check(sg.sg_orthogonalize(u.t()), u.t().contiguous())  # columns apart: copied


def test_empty():
    need_gpu()
    for shape in ((0, 4), (4, 0), (0, 3, 3), (2, 0, 3)):
        assert sg.sg_orthogonalize(torch.zeros(shape, device="cuda")).shape == shape


def test_same_bits_streams_and_graph():
    need_gpu()
    for dtype in ("bf16", "f32"):
        for shape in ((2, 100, 200), (300, 90)):
            u = make(shape, dtype)
            want = sg.sg_orthogonalize(u)
            B, (m, n) = (shape[0] if len(shape) == 3 else 1), shape[-2:]
            need = sg.lib().sg_orthogonalize_workspace_bytes(B, m, n, 1 if dtype == "bf16" else 0)
            ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got = sg.sg_orthogonalize(u, workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(got, want)
            graph = torch.cuda.CUDAGraph()
            su = u.clone()
            with torch.cuda.graph(graph):
                cap = sg.sg_orthogonalize(su)
            for seed in range(4):
                nu = make(shape, dtype, seed + 10)
                su.copy_(nu)
                graph.replay()
                eager = sg.sg_orthogonalize(nu)
                torch.cuda.synchronize()
                assert torch.equal(eager, cap)
