"""The operators around a step without a GPU: every host-checkable bad argument
is refused with the documented status before any launch, the binding refuses
tensors that do not fit, and the 64-bit definitions agree with automatic
differentiation and with a decomposition."""
import ctypes as C

import pytest
import torch

import sparse_gradient_synchronization_amd as sg
import step_ref as ref

SG_OK, SG_EINVAL, SG_ECAPACITY, SG_EUNSUPPORTED = 0, -1, -2, -5
F, G, N = C.c_void_p(0x10000), C.c_void_p(0x20000), None  # pointers that no host check dereferences
ODD = C.c_void_p(0x10001)
BIG = 1 << 45
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return sg.lib()


def make(L, fn, order, base):
    def f(**kw):
        a = dict(base, **kw)
        return getattr(L, fn)(*[a[k] for k in order])
    return f


def linear_ce(L):
    return make(L, "sg_linear_ce_loss", ("x", "ldx", "w", "ldw", "dt", "T", "V", "H", "it", "label", "weight", "zc", "loss", "lse",
                                         "gx", "ldgx", "gw", "ldgw", "keep", "ws", "nws", "stream"),
                dict(x=F, ldx=64, w=F, ldw=64, dt=1, T=8, V=100, H=64, it=1.0, label=F, weight=N, zc=0.0, loss=F, lse=F, gx=F,
                     ldgx=64, gw=G, ldgw=64, keep=1 << 20, ws=F, nws=BIG, stream=N))


def balance(L):
    return make(L, "sg_balance_loss", ("x", "dt", "T", "E", "ld", "idx", "k", "live", "alpha", "zc", "loss", "counts", "prob", "grad",
                                       "ldg", "ws", "nws", "stream"),
                dict(x=F, dt=0, T=8000, E=16, ld=16, idx=F, k=2, live=N, alpha=0.1, zc=0.1, loss=F, counts=F, prob=F, grad=G, ldg=16,
                     ws=F, nws=BIG, stream=N))


def ortho(L):
    return make(L, "sg_orthogonalize", ("x", "dt", "B", "m", "n", "ld", "stride", "steps", "a", "b", "c", "eps", "out", "ldo", "so",
                                        "ws", "nws", "stream"),
                dict(x=F, dt=0, B=2, m=16, n=24, ld=24, stride=384, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, out=G,
                     ldo=24, so=384, ws=F, nws=BIG, stream=N))


def test_linear_ce_arguments(L):
    f = linear_ce(L)
    for bad in (dict(dt=2), dict(V=0), dict(V=1 << 31), dict(H=0), dict(T=1 << 31), dict(ldx=63), dict(ldw=63), dict(ldgx=63),
                dict(ldgw=63), dict(ldx=1 << 40), dict(ldw=1 << 40), dict(ldgx=1 << 40), dict(ldgw=1 << 40), dict(x=N), dict(w=N),
                dict(label=N), dict(loss=N), dict(x=ODD), dict(w=ODD), dict(gx=ODD), dict(gw=ODD), dict(gw=F), dict(ws=N),
                dict(dt=0, x=C.c_void_p(0x10002))):
        assert f(**bad) == SG_EINVAL, bad
    for it in (0.0, -1.0, NAN, INF, 2e6, 1e-38):
        assert f(it=it) == SG_EINVAL
    for zc in (-1.0, NAN, INF, 2e6):
        assert f(zc=zc) == SG_EINVAL
    assert f(H=(1 << 20) + 8, ldx=1 << 21, ldw=1 << 21, ldgx=1 << 21, ldgw=1 << 21) == SG_EUNSUPPORTED
    assert f(T=(1 << 24) + 1) == SG_EUNSUPPORTED
    assert f(T=1 << 24, V=1 << 30) == SG_EUNSUPPORTED
    # grids of 2^32 threads: rows of long hidden states, logits in tiles of 128 x 128
    long = dict(H=4096, ldx=4096, ldw=4096, ldgx=4096, ldgw=4096)
    assert f(T=1 << 22, **long) == SG_EUNSUPPORTED and f(T=1 << 19, V=(1 << 19) + 1) == SG_EUNSUPPORTED
    assert f(T=(1 << 22) - 1, nws=0, **long) == SG_ECAPACITY and f(T=1 << 19, V=1 << 18, nws=0) == SG_ECAPACITY
    assert f(nws=0) == SG_ECAPACITY
    assert f(T=0, x=N, label=N, loss=N, gw=N) == SG_OK


def test_linear_ce_workspace(L):
    def need(T, V, H, dt=1, p=0x10000, ld=None, gx=1, gw=1, keep=1 << 40):
        return L.sg_linear_ce_workspace_bytes(T, V, H, dt, C.c_void_p(p), H if ld is None else ld, gx, gw, keep)
    f = linear_ce(L)
    full = need(512, 10000, 128)
    assert full >= 512 * 10000 * 2
    assert need(512, 10000, 128, keep=1 << 20) < full  # pieces
    assert need(512, 10000, 128, gx=0, gw=0, keep=0) < need(512, 10000, 128, keep=0)
    assert need(512, 10000, 127) > 10000 * 127 * 2 + need(512, 10000, 128, gx=0, gw=0)  # a copy of the head
    assert need(512, 10000, 128, p=0x10008) > full and need(512, 10000, 128, ld=132) > full
    assert need(0, 10, 10) == 0 and need(1, 0, 10) == 0
    assert f(T=512, V=10000, H=128, ldx=128, ldw=128, ldgx=128, ldgw=128, keep=1 << 40, nws=full - 1) == SG_ECAPACITY


def test_balance_arguments(L):
    f = balance(L)
    for bad in (dict(dt=2), dict(E=0), dict(k=0), dict(T=1 << 31), dict(ld=15), dict(ldg=15), dict(ld=1 << 40), dict(ldg=1 << 40),
                dict(x=N), dict(idx=N), dict(loss=N), dict(counts=N), dict(prob=N), dict(ws=N), dict(x=ODD), dict(grad=ODD),
                dict(grad=F, ldg=17), dict(alpha=-1.0), dict(alpha=NAN), dict(alpha=2e6), dict(zc=-1.0), dict(zc=NAN), dict(zc=INF)):
        assert f(**bad) == SG_EINVAL, bad
    assert f(E=1025, ld=1025, ldg=1025) == SG_EUNSUPPORTED
    assert f(k=17) == SG_EUNSUPPORTED
    assert f(T=1 << 30, k=2) == SG_EUNSUPPORTED
    assert f(nws=0) == SG_ECAPACITY


def test_orthogonalize_arguments(L):
    f = ortho(L)
    for bad in (dict(dt=2), dict(steps=0), dict(steps=65), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(a=NAN), dict(b=INF),
                dict(c=-INF), dict(ld=23), dict(ldo=23), dict(ld=1 << 40), dict(ldo=1 << 40), dict(stride=383), dict(so=383),
                dict(x=N), dict(out=N), dict(ws=N), dict(x=ODD), dict(out=ODD), dict(out=F, ldo=25, so=400), dict(out=F, so=400)):
        assert f(**bad) == SG_EINVAL, bad
    # coefficients whose iterates leave the scales' range
    for bad in (dict(a=5.0), dict(a=3.0, b=3.0, c=3.0), dict(b=-200.0), dict(a=1.0, b=0.0, c=60.0)):
        assert f(**bad) == SG_EUNSUPPORTED, bad
    assert f(B=1 << 16) == SG_EUNSUPPORTED
    assert f(n=1 << 21, ld=1 << 21, ldo=1 << 21, stride=1 << 26, so=1 << 26) == SG_EUNSUPPORTED
    assert f(nws=0) == SG_ECAPACITY
    for empty in (dict(B=0), dict(m=0), dict(n=0)):
        assert f(x=N, out=N, ws=N, **empty) == SG_OK


def test_workspace_sizes(L):
    one, two = L.sg_orthogonalize_workspace_bytes(1, 100, 200, 1), L.sg_orthogonalize_workspace_bytes(1, 100, 200, 0)
    assert 0 < one < two <= 2 * one + 4096
    assert L.sg_orthogonalize_workspace_bytes(1, 200, 100, 0) == two
    assert L.sg_orthogonalize_workspace_bytes(0, 1, 1, 0) == 0 and L.sg_orthogonalize_workspace_bytes(1, 1 << 21, 1, 0) == 0
    assert L.sg_balance_workspace_bytes(10000, 64, 2, 0) > 0 and L.sg_balance_workspace_bytes(10000, 1025, 2, 0) == 0
    assert L.sg_balance_workspace_bytes(10, 64, 2, 0) == 0  # one block needs none


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 8)
    for f in (lambda: sg.sg_linear_ce_loss(x, x, torch.zeros(4, dtype=torch.int32)),
              lambda: sg.sg_balance_loss(x, torch.zeros((4, 1), dtype=torch.int32)), lambda: sg.sg_orthogonalize(x)):
        with pytest.raises((ValueError, RuntimeError)):
            f()


def test_definitions_against_autograd():
    g = torch.Generator().manual_seed(0)
    x, w = (torch.randn(s, generator=g).double() for s in ((9, 5), (13, 5)))
    label = torch.tensor([0, 12, -1, 5, 5, 13, 2, 7, 1], dtype=torch.int32)
    weight = torch.rand(9, generator=g)
    weight[3] = 0
    a, b = x.float().requires_grad_(), w.float().requires_grad_()
    z = 0.7 * a.double() @ b.double().t()
    lse = torch.logsumexp(z, 1)
    live = (label >= 0) & (label < 13) & (weight != 0)
    loss = torch.where(live, weight.double() * (lse - z.gather(1, torch.where(live, label, 0).long()[:, None])[:, 0] + 0.1 * lse ** 2), 0.0)
    loss.sum().backward()
    val, _ = ref.linear_ce(a.detach(), b.detach(), label, weight, 0.7, 0.1)
    assert torch.allclose(val["loss"], loss.detach())
    assert torch.allclose(val["grad_hidden"], a.grad.double(), atol=1e-6) and torch.allclose(val["grad_head"], b.grad.double(), atol=1e-6)
    x = torch.randn((20, 6), generator=g).requires_grad_()
    idx = torch.topk(x.detach(), 2, dim=1).indices.int()
    live = torch.arange(20) % 3 != 0
    p = torch.softmax(x.double(), 1)[live]
    f = torch.bincount(idx[live].reshape(-1).long(), minlength=6).double() / idx[live].numel()
    loss = 0.3 * 6 * (f * p.mean(0)).sum() + 0.2 * torch.logsumexp(x.double(), 1)[live].square().mean()
    loss.backward()
    val, _ = ref.balance(x.detach(), idx, live, 0.3, 0.2)
    assert torch.allclose(val["loss"], loss.detach()) and torch.allclose(val["grad"], x.grad.double(), atol=1e-6)


@pytest.mark.parametrize("shape", [(7, 12), (12, 7), (2, 5, 5)])
def test_definition_against_decomposition(shape):
    u = torch.randn(shape, generator=torch.Generator().manual_seed(1))
    p, s, q = torch.linalg.svd(u.double(), full_matrices=False)
    t = s / (s.square().sum(-1, keepdim=True).sqrt() + 1e-7)
    a, b, c = 3.4445, -4.7750, 2.0315
    for _ in range(5):
        t = a * t + b * t ** 3 + c * t ** 5
    assert torch.allclose(ref.orthogonalize(u, 5, (a, b, c), 1e-7), (p * t[..., None, :]) @ q)
