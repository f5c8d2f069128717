"""The vocabulary operators without a GPU: every host-checkable bad argument
is refused with the documented status before any launch, the binding refuses
tensors that do not fit, and the 64-bit definitions agree with each other."""
import ctypes as C

import numpy as np
import pytest
import torch

import rowloss_ref as ref
import sparse_gradient_synchronization_amd as sg

SG_OK, SG_EINVAL, SG_ECAPACITY, SG_EUNSUPPORTED = 0, -1, -2, -5
F, N = C.c_void_p(0x10000), None  # F: a non-null pointer that no host check dereferences
ODD = C.c_void_p(0x10001)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    return sg.lib()


def calls(L):
    """name -> f(**changes): the call with valid arguments but for the changed ones."""
    def make(fn, order, base):
        def f(**kw):
            a = dict(base, **kw)
            return getattr(L, fn)(*[a[k] for k in order])
        return f

    rows = dict(x=F, dt=0, T=4, V=1000, ld=1000, it=1.0, ws=F, nws=BIG, stream=N, grad=F, ldg=1000, weight=N)
    return {
        "topk": make("sg_topk_rows", ("x", "dt", "T", "V", "ld", "it", "k", "idx", "logp", "lse", "ws", "nws", "stream"),
                     dict(rows, k=8, idx=F, logp=F, lse=N)),
        "distill": make("sg_distill_loss", ("x", "dt", "T", "V", "ld", "it", "idx", "logp", "k", "mode", "weight", "loss",
                                            "grad", "ldg", "ws", "nws", "stream"),
                        dict(rows, k=8, idx=F, logp=F, mode=2, loss=F)),
        "policy": make("sg_policy_loss", ("x", "dt", "T", "V", "ld", "it", "action", "old", "ref", "adv", "weight", "lo",
                                          "hi", "kl", "loss", "logp", "grad", "ldg", "ws", "nws", "stream"),
                       dict(rows, action=F, old=F, ref=F, adv=F, lo=0.2, hi=0.2, kl=0.1, loss=F, logp=N)),
        "preference": make("sg_preference_loss", ("x", "dt", "T", "V", "ld", "label", "off", "pairs", "ref", "weight",
                                                  "kind", "beta", "eps", "average", "loss", "logp", "grad", "ldg", "ws",
                                                  "nws", "stream"),
                           dict(rows, label=F, off=F, pairs=2, ref=N, kind=0, beta=0.1, eps=0.0, average=0, loss=F,
                                logp=N)),
    }


ALL = ["topk", "distill", "policy", "preference"]


@pytest.mark.parametrize("op", ALL)
def test_row_arguments(L, op):
    f = calls(L)[op]
    nan = float("nan")
    for bad in (dict(dt=2), dict(dt=-1), dict(V=0), dict(V=1 << 31, ld=1 << 31, ldg=1 << 31), dict(T=1 << 31),
                dict(ld=999), dict(ld=1 << 40), dict(x=N), dict(x=ODD), dict(x=C.c_void_p(0x10002))):
        assert f(**bad) == SG_EINVAL, bad
    if op != "preference":
        for it in (0.0, -1.0, nan, float("inf"), 2e6):
            assert f(it=it) == SG_EINVAL, it
        assert f(T=0, x=N) == SG_OK
    if op != "topk":
        for bad in (dict(ldg=999), dict(ldg=1 << 40), dict(grad=ODD), dict(grad=F, x=F, ldg=1001)):
            assert f(**bad) == SG_EINVAL, bad
        assert f(loss=N) == SG_EINVAL


def test_topk_arguments(L):
    f = calls(L)["topk"]
    for bad in (dict(k=0), dict(k=1001), dict(idx=N), dict(logp=N)):
        assert f(**bad) == SG_EINVAL, bad
    assert f(V=5000, ld=5000, k=1025) == SG_EUNSUPPORTED


def test_distill_arguments(L):
    f = calls(L)["distill"]
    for bad in (dict(k=0), dict(idx=N), dict(logp=N), dict(mode=3), dict(mode=-1)):
        assert f(**bad) == SG_EINVAL, bad
    assert f(k=1025) == SG_EUNSUPPORTED


def test_policy_arguments(L):
    f = calls(L)["policy"]
    nan = float("nan")
    for bad in (dict(action=N), dict(lo=-0.1), dict(lo=1.1), dict(lo=nan), dict(hi=-0.1), dict(hi=nan), dict(hi=2e6),
                dict(kl=-0.1), dict(kl=nan), dict(kl=2e6)):
        assert f(**bad) == SG_EINVAL, bad


def test_preference_arguments(L):
    f = calls(L)["preference"]
    nan = float("nan")
    for bad in (dict(label=N), dict(off=N), dict(kind=3), dict(kind=-1), dict(beta=0.0), dict(beta=nan), dict(beta=-1.0),
                dict(eps=-0.1), dict(eps=0.5), dict(eps=nan), dict(kind=1, eps=0.1), dict(pairs=1 << 30), dict(ws=N)):
        assert f(**bad) == SG_EINVAL, bad
    need = L.sg_preference_workspace_bytes(4, 1000, 0)
    assert need >= 4 * (8 + 3 * 4)
    assert f(nws=need - 1) == SG_ECAPACITY


def test_workspaces(L):
    """Few long rows are split and need room for their parts; sizes out of range have none."""
    assert L.sg_preference_workspace_bytes(1 << 31, 1000, 0) == 0
    assert L.sg_preference_workspace_bytes(100, 0, 0) == 0
    for T in (1, 3, 100, 5000):
        for V in (1, 1000, 131072, 1 << 20):
            for dt in (0, 1):
                for need, call in ((L.sg_topk_rows_workspace_bytes(T, V, 1, dt), dict(k=1)),):
                    if need:
                        assert calls(L)["topk"](T=T, V=V, ld=V, dt=dt, nws=need - 1, **call) == SG_ECAPACITY
                        assert calls(L)["topk"](T=T, V=V, ld=V, dt=dt, ws=N, **call) == SG_EINVAL
                need = L.sg_distill_workspace_bytes(T, V, 4, dt)
                if need:
                    assert calls(L)["distill"](T=T, V=V, ld=V, ldg=V, dt=dt, nws=need - 1, k=4) == SG_ECAPACITY
                    assert calls(L)["distill"](T=T, V=V, ld=V, ldg=V, dt=dt, ws=N, k=4) == SG_EINVAL
                need = L.sg_policy_workspace_bytes(T, V, dt)
                if need:
                    assert calls(L)["policy"](T=T, V=V, ld=V, ldg=V, dt=dt, nws=need - 1) == SG_ECAPACITY
                    assert calls(L)["policy"](T=T, V=V, ld=V, ldg=V, dt=dt, ws=N) == SG_EINVAL


def test_binding_refuses():
    x = torch.zeros(4, 16)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: sg.sg_topk_rows(x, 2), lambda: sg.sg_distill_loss(x, i, i.float()),
                 lambda: sg.sg_policy_loss(x, i[:, 0]),
                 lambda: sg.sg_preference_loss(x, i[:, 0], torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        sg._rows(torch.zeros(4, 5, 6))
    with pytest.raises(TypeError):
        sg._rows(torch.zeros(4, 5, dtype=torch.float16))
    with pytest.raises(ValueError):
        sg._beside(x, "weight", torch.zeros(5), torch.float32, (4,))
    with pytest.raises(ValueError):
        sg._beside(x, "weight", torch.zeros(4, dtype=torch.float64), torch.float32, (4,))
    with pytest.raises(ValueError):
        sg._grad_of(x, True, torch.zeros(4, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        sg._grad_of(x, True, torch.zeros(16, 4).t())
    for temperature in (0.0, -1.0, float("nan")):
        with pytest.raises(ValueError):
            sg._inv_temp(temperature)


def test_rows_takes_strided_rows_as_they_are():
    buf = torch.zeros(4, 20)
    x, dt, T, V, ld = sg._rows(buf[:, 3:16])
    assert x.data_ptr() == buf.data_ptr() + 12 and (dt, T, V, ld) == (0, 4, 13, 20)
    x, _, T, V, ld = sg._rows(torch.zeros(6, 4).t())
    assert x.is_contiguous() and (T, V, ld) == (4, 6, 6)
    x, _, T, V, ld = sg._rows(torch.zeros(1, 6).expand(4, 6))
    assert x.is_contiguous() and ld == 6


# ---------------------------------------------------------------------------
# the 64-bit definitions against each other
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("mode", ["plain", "renorm", "tail"])
def test_distill_definition_against_differences(mode):
    rng = np.random.default_rng(1)
    x = rng.normal(0, 1.5, 30)
    idx = rng.permutation(30)[:9]
    logp = np.log(rng.dirichlet(np.ones(9)) * 0.8)
    _, g, _ = ref.distill_row(x, idx, logp, 0.7, mode)
    for i in range(30):
        h = np.zeros(30)
        h[i] = 1e-5
        d = (ref.distill_row(x + h, idx, logp, 0.7, mode)[0] - ref.distill_row(x - h, idx, logp, 0.7, mode)[0]) / 2e-5
        assert abs(d - g[i]) < 1e-8


def test_distill_definition_is_a_divergence():
    """With the whole vocabulary listed the three modes are the plain divergence, and zero for equal distributions."""
    rng = np.random.default_rng(2)
    x, y = rng.normal(0, 1, 20), rng.normal(0, 1, 20)
    lp = ref.log_softmax(y, 1.0)[0]
    kl = (np.exp(lp) * (lp - ref.log_softmax(x, 1.0)[0])).sum()
    for mode in ("plain", "renorm", "tail"):
        assert abs(ref.distill_row(x, np.arange(20), lp, 1.0, mode)[0] - kl) < 1e-12
        assert abs(ref.distill_row(y, np.arange(20), lp, 1.0, mode)[0]) < 1e-12


def test_policy_and_preference_definitions_against_differences():
    rng = np.random.default_rng(3)
    for old, adv in ((-1.0, 1.0), (-4.0, 1.0), (-1.0, -1.0), (-9.0, -1.0)):
        x = rng.normal(0, 1, 12)
        args = (3, old, -2.0, adv, 1.3, 0.2, 0.3, 0.1)
        g = ref.policy_row(x, *args)[2]
        for i in range(12):
            h = np.zeros(12)
            h[i] = 1e-5
            d = (ref.policy_row(x + h, *args)[0] - ref.policy_row(x - h, *args)[0]) / 2e-5
            assert abs(d - g[i]) < 1e-8 * max(1.0, abs(d))
    x = rng.normal(0, 1, (6, 8))
    for kind in ("sigmoid", "hinge", "ipo"):
        args = (np.array([1, 2, -1, 7, 0, 3]), np.array([0, 1, 3, 4, 6]), rng.normal(0, 1, 4), np.array([1.0, 0.5]),
                kind, 0.3, 0.1 if kind == "sigmoid" else 0.0, True)
        g = ref.preference(x, *args)[2]
        for t in range(6):
            for i in range(8):
                h = np.zeros((6, 8))
                h[t, i] = 1e-5
                d = (ref.preference(x + h, *args)[0].sum() - ref.preference(x - h, *args)[0].sum()) / 2e-5
                assert abs(d - g[t, i]) < 1e-8
