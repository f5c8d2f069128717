"""The head's cross entropy against its definition in 64 bits."""
import pytest
import torch

import sparse_gradient_synchronization_amd as sg
import step_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ("loss", "lse", "grad_hidden", "grad_head")


def make(T, V, H, dtype, seed=0, masked=0.2, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    w = (torch.randn((V, H), device="cuda", generator=g) * scale / H ** 0.5).to(DT[dtype])
    label = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    lift = 3 * torch.rand((T, 1), device="cuda", generator=g)
    x = (torch.randn((T, H), device="cuda", generator=g) + lift * w[label.long()].float()).to(DT[dtype])
    label[torch.rand(T, device="cuda", generator=g) < masked] = -100
    weight = torch.rand(T, device="cuda", generator=g) + 0.25
    return x, w, label, weight


def check(out, x, w, label, weight, it=1.0, zc=0.0):
    val, err = ref.linear_ce(x, w, label, weight, it, zc)
    for name, got in zip(NAMES, out):
        if got is not None:
            ref.close(got, val[name], err[name], name)
    assert sg.sg_device_error() == 0


# one row, one token, one column; tiles' edges (32, 128, 256) and odd sizes on
# every side; few, some and many rows
SIZES = [(1, 1, 1), (1, 7, 3), (2, 300, 64), (31, 129, 65), (32, 128, 128), (33, 257, 100), (64, 1000, 72),
         (65, 255, 8), (128, 512, 192), (129, 1111, 129), (300, 4097, 264), (1030, 257, 63), (17, 20001, 40)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,H", SIZES)
def test_sizes(T, V, H, dtype):
    need_gpu()
    x, w, label, weight = make(T, V, H, dtype, T + V)
    out = sg.sg_linear_ce_loss(x, w, label, weight=weight, temperature=0.8, z_coef=1e-3)
    check(out, x, w, label, weight, 1.25, 1e-3)
    # as few exponentials kept as can be: the vocabulary in pieces of 256
    out = sg.sg_linear_ce_loss(x, w, label, weight=weight, temperature=0.8, z_coef=1e-3, keep_bytes=0)
    check(out, x, w, label, weight, 1.25, 1e-3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_tiles(dtype):
    """Enough rows and tokens for the largest tile of every product."""
    need_gpu()
    for T, V, H in [(4100, 4100, 256), (520, 33000, 136)]:
        x, w, label, weight = make(T, V, H, dtype, 5)
        check(sg.sg_linear_ce_loss(x, w, label, weight=weight), x, w, label, weight)
        out = sg.sg_linear_ce_loss(x, w, label, weight=weight, keep_bytes=4 * T * 1500)
        check(out, x, w, label, weight)


# The variants that a rule on sizes chooses, at both sides of each rule's edge: dw as a stream of rows (64 rows)
# with the hidden dimension in parts or whole, dw in parts of the rows, dx in many parts of the vocabulary, rows found
# by the blocks that pack them (1024), statistics joined in the pass to g (32 tiles of columns)
VARIANTS = [(1023, 4096, 40), (1024, 4097, 40), (1025, 4096, 40), (50, 8192, 72), (50, 8193, 72),
            (63, 700, 700), (64, 700, 257), (65, 700, 257), (3, 130, 2056), (40, 70000, 65), (4088, 3264, 64),
            (6000, 150, 96), (200, 40000, 60), (1100, 300, 1030)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,H", VARIANTS)
def test_variants(T, V, H, dtype):
    """Into rows apart that start on 16 bytes and into rows that start anywhere."""
    need_gpu()
    x, w, label, weight = make(T, V, H, dtype, T)
    out = sg.sg_linear_ce_loss(x, w, label, weight=weight)
    check(out, x, w, label, weight)
    for pad in (16 - H % 8, 1):
        flat = torch.full((V * (H + pad) + 3,), 7.0, device="cuda", dtype=x.dtype)
        gw = flat[int(pad == 1):][:V * (H + pad)].view(V, H + pad)
        sg.sg_linear_ce_loss(x, w, label, weight=weight, grad_head=gw[:, :H])
        assert torch.equal(gw[:, :H], out[3]) and bool((gw[:, H:] == 7.0).all()) and bool((flat[-2:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_outputs_alone(dtype):
    """Each gradient alone, none, and the loss the same bits whatever is asked for."""
    need_gpu()
    x, w, label, weight = make(200, 900, 96, dtype)
    full = sg.sg_linear_ce_loss(x, w, label, weight=weight)
    check(full, x, w, label, weight)
    none = sg.sg_linear_ce_loss(x, w, label, weight=weight, want_grad=False)
    assert none[2] is None and none[3] is None
    gx, gw = torch.empty_like(x), torch.empty_like(w)
    only_x = sg.sg_linear_ce_loss(x, w, label, weight=weight, want_grad=False, grad_hidden=gx)
    only_w = sg.sg_linear_ce_loss(x, w, label, weight=weight, want_grad=False, grad_head=gw)
    assert only_x[3] is None and only_w[2] is None
    for o in (none, only_x, only_w):
        assert torch.equal(o[0], full[0]) and torch.equal(o[1], full[1])
    assert torch.equal(gx, full[2]) and torch.equal(gw, full[3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_places(dtype):
    """Rows apart, matrices that start anywhere, gradients into the middle of
    larger buffers (whose rest stays), the hidden states' gradient over them."""
    need_gpu()
    for off, pad in [(1, 7), (3, 8), (8, 24), (0, 1)]:
        T, V, H = 70, 700, 90
        x, w, label, weight = make(T, V, H, dtype, off)
        bx = torch.full((T + 1, H + pad), float("nan"), device="cuda", dtype=x.dtype).reshape(-1)
        bw = torch.full((V + 1, H + pad), float("nan"), device="cuda", dtype=x.dtype).reshape(-1)
        vx = bx[off:off + T * (H + pad)].view(T, H + pad)[:, :H]
        vw = bw[off:off + V * (H + pad)].view(V, H + pad)[:, :H]
        vx.copy_(x), vw.copy_(w)
        gbx, gbw = torch.full_like(bx, 7.0), torch.full_like(bw, 7.0)
        gx = gbx[off:off + T * (H + pad)].view(T, H + pad)[:, :H]
        gw = gbw[off:off + V * (H + pad)].view(V, H + pad)[:, :H]
        out = sg.sg_linear_ce_loss(vx, vw, label, weight=weight, grad_hidden=gx, grad_head=gw)
        check(out, x, w, label, weight)
        for b, v in ((gbx, gx), (gbw, gw)):
            rest = torch.ones_like(b, dtype=torch.bool)
            rest[off:off + v.shape[0] * (H + pad)].view(-1, H + pad)[:, :H] = False
            assert bool((b[rest] == 7.0).all())
        out2 = sg.sg_linear_ce_loss(vx, vw, label, weight=weight, grad_hidden=vx, grad_head=gw)
        assert torch.equal(vx, gx) and torch.equal(out2[0], out[0])
    # a transposed head is copied
    x, w, label, weight = make(40, 64, 64, dtype)
    check(sg.sg_linear_ce_loss(x, w.t().contiguous().t(), label, weight=weight), x, w, label, weight)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_do_not_count(dtype):
    """Labels outside, weights of 0: never read, whatever they hold; all rows; no rows."""
    need_gpu()
    x, w, label, weight = make(130, 600, 64, dtype, masked=0.0)
    label[::3] = 600
    label[1::7] = -1
    label[5] = 2 ** 31 - 1
    weight[4::9] = 0.0
    dead = (label < 0) | (label >= 600) | (weight == 0)
    x[dead] = float("nan")
    out = sg.sg_linear_ce_loss(x, w, label, weight=weight)
    clean = torch.where(dead[:, None], torch.zeros_like(x), x)
    check(out, clean, w, label, weight)
    assert bool((out[2][dead] == 0).all()) and bool((out[0][dead] == 0).all()) and bool((out[1][dead] == 0).all())
    for lab in (torch.full_like(label, -100), label):
        z = sg.sg_linear_ce_loss(x, w, lab, weight=torch.zeros_like(weight))
        for t in z:
            assert bool((t == 0).all())
    empty = sg.sg_linear_ce_loss(x[:0], w, label[:0], grad_head=torch.full_like(w, 5.0))
    assert empty[0].shape == (0,) and bool((empty[3] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_not_finite(dtype):
    """A NaN or infinity of one row stays in its row's loss and gradient, and reaches the whole
    head's gradient; one in the head reaches everything."""
    need_gpu()
    x, w, label, weight = make(70, 300, 64, dtype, masked=0.0)
    ok = sg.sg_linear_ce_loss(x, w, label, weight=weight)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[3, 5] = bad
        out = sg.sg_linear_ce_loss(y, w, label, weight=weight)
        rest = torch.arange(70, device="cuda") != 3
        assert bool(out[0][3].isnan()) and bool(out[2][3].isnan().all()) and bool(out[3].isnan().any())
        assert not bool(out[0][rest].isnan().any()) and not bool(out[2][rest].isnan().any())
        if dtype == "bf16":
            assert torch.equal(out[2][rest], ok[2][rest])
    v = w.clone()
    v[7, 2] = float("nan")
    out = sg.sg_linear_ce_loss(x, v, label, weight=weight)
    assert bool(out[0].isnan().all()) and bool(out[2].isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["hidden", "weight"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_row_not_finite_leaves_the_others_their_precision(bad, where, dtype):
    """The other rows against their definition, small operands among them."""
    need_gpu()
    x, w, label, weight = make(50, 700, 64, dtype, masked=0.0, scale=1e-3)
    x = (x.float() * 1e-4).to(x.dtype)
    lone = label.clone()
    lone[20] = -100
    val, err = ref.linear_ce(x, w, lone, weight, 1.0, 0.0)
    if where == "hidden":
        x[20, 11] = bad
    else:
        weight[20] = bad
    out = sg.sg_linear_ce_loss(x, w, label, weight=weight)
    rest = torch.arange(50, device="cuda") != 20
    for name, got in zip(NAMES[:3], out):
        ref.close(got[rest], val[name][rest], err[name][rest], name)
    assert not bool(out[0][20].isfinite()) and not bool(out[2][20].isfinite().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-30, 1e-6, 0.0, 300.0, 1e15])
def test_magnitudes(scale, dtype):
    """Tiny and large operands: a constant softmax, and one that is a single token."""
    need_gpu()
    x, w, label, weight = make(50, 400, 64, dtype)
    w = (w.float() * scale).to(w.dtype)
    x = (x.float() / (1e15 if scale == 1e15 else 1.0)).to(x.dtype)
    check(sg.sg_linear_ce_loss(x, w, label, weight=weight), x, w, label, weight)


def test_weights_far_apart():
    """Weights over 2^20, negative ones, one for all; the rows with little keep their gradients."""
    need_gpu()
    for dtype in ("bf16", "f32"):
        x, w, label, weight = make(60, 500, 64, dtype)
        weight = weight * 2.0 ** -(torch.arange(60, device="cuda") % 20).float()
        weight[::5] *= -1
        check(sg.sg_linear_ce_loss(x, w, label, weight=weight), x, w, label, weight)
        check(sg.sg_linear_ce_loss(x, w, label), x, w, label, None)
        tiny = weight * 1e-30
        check(sg.sg_linear_ce_loss(x, w, label, weight=tiny), x, w, label, tiny)


def test_same_bits_again_and_dirty_workspace():
    need_gpu()
    for dtype in ("bf16", "f32"):
        for T, V, H, keep in [(100, 3000, 200, 1 << 30), (100, 3000, 200, 0), (20, 900, 64, 1 << 30)]:
            x, w, label, weight = make(T, V, H, dtype)
            a = sg.sg_linear_ce_loss(x, w, label, weight=weight, keep_bytes=keep)
            dt = 1 if dtype == "bf16" else 0
            need = sg.lib().sg_linear_ce_workspace_bytes(T, V, H, dt, w.data_ptr(), H, 1, 1, keep)
            ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
            b = sg.sg_linear_ce_loss(x, w, label, weight=weight, keep_bytes=keep, workspace=ws)
            for p, q in zip(a, b):
                assert torch.equal(p, q)


def test_streams_and_graph():
    """On another stream, and captured: replays on changed inputs equal eager calls."""
    need_gpu()
    for dtype in ("bf16", "f32"):
        x, w, label, weight = make(90, 1500, 128, dtype)
        want = sg.sg_linear_ce_loss(x, w, label, weight=weight)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = sg.sg_linear_ce_loss(x, w, label, weight=weight)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        graph = torch.cuda.CUDAGraph()
        sx, sl = x.clone(), label.clone()
        with torch.cuda.graph(graph):
            cap = sg.sg_linear_ce_loss(sx, w, sl, weight=weight)
        for seed in range(4):
            nx, _, nl, _ = make(90, 1500, 128, dtype, seed, masked=0.1 * seed)
            sx.copy_(nx), sl.copy_(nl)
            graph.replay()
            eager = sg.sg_linear_ce_loss(nx, w, nl, weight=weight)
            torch.cuda.synchronize()
            for a, b in zip(eager, cap):
                assert torch.equal(a, b)


def test_gradients_against_differences():
    """Central differences of the 64-bit loss along random directions."""
    need_gpu()
    x, w, label, weight = make(40, 300, 48, "f32")
    out = sg.sg_linear_ce_loss(x, w, label, weight=weight, z_coef=0.01)
    g = torch.Generator(device="cuda").manual_seed(9)
    for which in (0, 1):
        d = torch.randn((x, w)[which].shape, device="cuda", generator=g, dtype=torch.float64)
        h = 1e-5
        f = [_loss64(x.double() + (s * h * d if which == 0 else 0.0), w.double() + (s * h * d if which else 0.0),
                     label, weight, 0.01) for s in (1, -1)]
        slope = float(f[0] - f[1]) / (2 * h)
        mine = float((out[2 + which].double() * d).sum())
        size = float((out[2 + which].double() * d).abs().sum())
        assert abs(slope - mine) <= 1e-6 * size + 1e-6 * abs(slope)


def _loss64(x, w, label, weight, zc):
    live = label >= 0
    z = x @ w.t()
    lse = torch.logsumexp(z, 1)
    zy = z.gather(1, label.clamp_min(0).long()[:, None])[:, 0]
    return (torch.where(live, weight.double(), 0.0) * (lse - zy + zc * lse ** 2)).sum()
