"""The vocabulary losses on batches of the sizes that training takes, every
kernel of the preference loss among them, against the definitions in 64 bits;
calls without a gradient; and sums whose small terms count."""
import numpy as np
import pytest
import torch

import rowloss_ref as ref
import sparse_gradient_synchronization_amd as sg
from gpu_util import need_gpu
from test_gpu_rowlimits import check_distill, distill_bounds, sum_bound
from test_gpu_rowloss import KINDS, MODES, TDT, check, dev, host, make_lists, make_logits, policy_inputs

pytestmark = pytest.mark.gpu


def gpu_logits(seed, T, V, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, V), device="cuda", generator=g) * 2
    x.scatter_(1, torch.randint(0, V, (T, 3), device="cuda", generator=g),
               3 + 6 * torch.rand((T, 3), device="cuda", generator=g))
    return x.to(TDT[dtype]), g


def within(got, want, tol, what):
    """check() on the GPU, for whole gradients."""
    off = (got - want).abs()
    bad = ~(off <= tol)
    n = int(bad.sum())
    assert n == 0, "%s: %d off, largest %r of tolerance" % (what, n, float((off / tol)[bad].max()))


# threads and kernels of a call: joint launch or three (T 1024, 256 pairs), a wave or
# 256 threads to a gradient row (4 KB), 256 or 1024 threads to a pair (2048 rows), stores past
# the caches (256 MB), more rows or pairs than a grid dimension
@pytest.mark.parametrize("T,V,pairs,dtype,kind,average", [
    (1024, 700, 256, "f32", "sigmoid", False), (1025, 700, 3, "f32", "sigmoid", False), (1500, 2047, 4, "bf16", "ipo", True),
    (1500, 5003, 3, "bf16", "hinge", False), (1300, 5003, 3, "f32", "ipo", True), (4200, 600, 2, "f32", "sigmoid", True),
    (4200, 3001, 2, "bf16", "ipo", True), (4096, 600, 2, "f32", "hinge", False), (2000, 900, 300, "f32", "sigmoid", False),
    (800, 900, 300, "bf16", "ipo", False), (1100, 131072, 4, "bf16", "sigmoid", True), (1030, 66048, 4, "f32", "ipo", True),
    (1100, 123011, 4, "bf16", "ipo", True), (65700, 130, 40, "f32", "sigmoid", False), (70500, 33, 70000, "f32", "sigmoid", False)])
def test_preference_batches(T, V, pairs, dtype, kind, average):
    need_gpu()
    x, g = gpu_logits(T + V, T, V, dtype)
    B, beta = pairs, 0.3
    rng = np.random.default_rng(T)
    off = np.sort(rng.integers(2, T - 1, 2 * B + 1))  # rows before the first sequence and after the last
    label = rng.integers(0, V, T)
    label[rng.random(T) < 0.2] = -1
    label[::97] = V
    w = np.linspace(0.4, 1.0, B).astype(np.float32)
    y = dev(np.where((label >= 0) & (label < V), label, 0), torch.int64)
    counts = dev((label >= 0) & (label < V), torch.float64)
    step = max(1, (1 << 26) // V)
    lp = torch.cat([torch.log_softmax(x[a:a + step].double(), 1).gather(1, y[a:a + step, None])[:, 0]
                    for a in range(0, T, step)]) * counts
    lens = torch.from_numpy(np.diff(off))
    inside = slice(int(off[0]), int(off[-1]))
    seq = torch.repeat_interleave(torch.arange(2 * B), lens)
    add = lambda v: torch.zeros(2 * B, dtype=torch.float64).index_add_(0, seq, v[inside].cpu()).cuda()  # noqa: E731
    n = add(counts)
    per = n.clamp_min(1.0) if average else torch.ones_like(n)
    S = add(lp) / per
    rf = (S.cpu() + torch.from_numpy(rng.normal(0, 2.0, 2 * B))).float()
    d = S - rf.cuda().double()
    d = d[:B] - d[B:]
    eps = 0.1 if kind == "sigmoid" else 0.0
    W = dev(w, torch.float64)
    if kind == "ipo":
        L, s = (d - 0.5 / beta) ** 2, 2 * (d - 0.5 / beta)
    elif kind == "hinge":
        L, s = (1 - beta * d).clamp_min(0), torch.where(beta * d < 1, -beta, 0.0)
    else:
        h = beta * d
        L = (1 - eps) * torch.nn.functional.softplus(-h) + eps * torch.nn.functional.softplus(h)
        s = beta * (eps * torch.sigmoid(h) - (1 - eps) * torch.sigmoid(-h))
    se = sum_bound(V)
    each = n / per * se  # error of a sequence's sum, and of their difference
    derr = each[:B] + each[B:]  # the sums stay in fp64
    bend = {"ipo": 2.0, "hinge": 0.0, "sigmoid": beta * beta}[kind]
    args = (dev(label, torch.int32), dev(off, torch.int64), rf.cuda(), dev(w, torch.float32))
    kw = dict(kind=KINDS[kind], beta=beta, smoothing=eps, average=average)
    loss, logp, grad = sg.sg_preference_loss(x, *args, **kw)
    within(logp.double(), S, each + 2.0 ** -24 * S.abs() + 1e-30, "sequence logp")
    within(loss.double(), W * L, W * (s.abs() + bend * derr) * derr + 2.0 ** -24 * (W * L).abs() + 1e-30, "loss")
    alone, logp_alone, none = sg.sg_preference_loss(x, *args, want_grad=False, **kw)
    assert none is None
    within(alone.double(), W * L, W * (s.abs() + bend * derr) * derr + 2.0 ** -24 * (W * L).abs() + 1e-30, "loss alone")
    within(logp_alone.double(), S, each + 2.0 ** -24 * S.abs() + 1e-30, "sequence logp alone")
    slope, slope_off = torch.zeros(T, dtype=torch.float64, device="cuda"), torch.zeros(T, dtype=torch.float64, device="cuda")
    slope[inside] = (torch.cat([W * s, -W * s]) / per)[seq.cuda()] * counts[inside]
    slope_off[inside] = (torch.cat([W * bend * derr] * 2) / per)[seq.cuda()] * counts[inside]
    for a in range(0, T, step):
        b = slice(a, a + step)
        xd = x[b].double()
        q = torch.softmax(xd, 1)
        depth = xd.amax(1, keepdim=True) - xd
        del xd
        toward = -q
        toward[torch.arange(q.shape[0]), y[b]] += 1.0
        want = slope[b, None] * toward
        tol = want.abs() * (2 * se + 2.0 ** -22 + 3 * 2.0 ** -24 * depth + ref.HALF[dtype])
        tol += slope_off[b, None] * toward.abs() + slope[b, None].abs() * q * 2 * se + 2.0 ** -126 * 4
        within(grad[b].double(), want, tol, "gradient of rows from %d" % a)
        if a == 0:
            assert not grad[:2].any()  # of no sequence
    z = x.clone()
    loss2, logp2, g2 = sg.sg_preference_loss(z, *args, grad=z, **kw)
    assert torch.equal(loss, loss2) and torch.equal(logp, logp2) and torch.equal(grad, g2)
    assert sg.sg_device_error() == 0


@pytest.mark.parametrize("T,V", [(5, 900), (300, 5003), (130, 33000), (4, 140001), (200, 66001)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_policy_without_gradient(T, V, dtype):
    need_gpu()
    temp = 0.8
    x, xs = make_logits(T + V, T, V, dtype)
    a, old, rf, adv = policy_inputs(V + 1, xs, 1.0 / temp)
    w = np.linspace(0.2, 1.0, T).astype(np.float32)
    w[1] = 0.0
    loss, logp, none = sg.sg_policy_loss(x, dev(a, torch.int32), dev(old, torch.float32), dev(adv, torch.float32),
                                         dev(rf, torch.float32), dev(w, torch.float32), 0.2, 0.28, 0.05, temp, want_grad=False)
    assert none is None
    L, P, tl, tp = np.zeros(T), np.zeros(T), np.zeros(T), np.zeros(T)
    for t in range(T):
        if w[t] == 0:
            continue
        l, p, _ = ref.policy_row(xs[t], a[t], float(old[t]), float(rf[t]), float(adv[t]), 1.0 / temp, 0.2, 0.28, 0.05)
        L[t], P[t] = w[t] * l, p
        # the temperature as fp32 rounds it moves a log-probability by half a unit of its distance from the row's mean
        far = abs(p) + np.log(V)
        e = sum_bound(V) + 2.0 ** -24 * far
        r = np.exp(p - float(old[t]))
        move = abs(r * adv[t]) + 0.05 * abs(1 - np.exp(rf[t] - p))
        bend = abs(r * adv[t]) + 0.05 * np.exp(rf[t] - p)
        tl[t] = w[t] * (move + bend * e) * e + 2.0 ** -24 * abs(L[t])
        tp[t] = e + 2.0 ** -24 * abs(p)
    check(host(logp), P, tp, "logp")
    check(host(loss), L, tl, "loss")


@pytest.mark.parametrize("dtype,V", [("bf16", 131072), ("f32", 66048), ("bf16", 123011)])
def test_distill_and_policy_gradients_beyond_the_cache(dtype, V):
    """More than 256 MB of gradient: stores past the caches where logits and gradient lie alike, ordinary ones elsewhere."""
    need_gpu()
    T, k = 1100, 24
    x, g = gpu_logits(V, T, V, dtype)
    idx, logp = make_lists(V, T, V, k)
    rows = [0, 1, 511, 777, T - 2, T - 1]
    loss, grad = sg.sg_distill_loss(x, dev(idx, torch.int32), dev(logp, torch.float32))
    L, G, tl, tg = distill_bounds(host(x[rows]), idx[rows], logp[rows], np.ones(len(rows)), 1.0, "tail")
    check(host(loss[rows]), L, tl, "loss")
    check(host(grad[rows]), G, tg + ref.HALF[dtype] * np.abs(G) + 2.0 ** -122, "gradient")
    action = torch.randint(0, V, (T,), device="cuda", generator=g)
    adv = torch.randn(T, device="cuda", generator=g)
    _, lp, grad = sg.sg_policy_loss(x, action.int(), None, adv)
    se = sum_bound(V)
    for a in range(0, T, 256):
        xd = x[a:a + 256].double()
        q = torch.softmax(xd, 1)
        toward = -q
        toward[torch.arange(q.shape[0]), action[a:a + 256]] += 1.0
        want = -adv[a:a + 256, None].double() * toward
        tol = want.abs() * (2 * se + 2.0 ** -22 + 3 * 2.0 ** -24 * (xd.amax(1, keepdim=True) - xd) + ref.HALF[dtype])
        tol += adv[a:a + 256, None].abs() * q * 2 * se + 2.0 ** -126 * 4
        within(grad[a:a + 256].double(), want, tol, "policy gradient of rows from %d" % a)


# ---------------------------------------------------------------------------
# sums
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(3, 1021), (3, 8000), (140, 30011), (2, 70001), (130, 131072)])
@pytest.mark.parametrize("depth", [16, 20])
def test_small_terms_of_a_sum_are_not_lost(depth, T, V, dtype):
    """One logit of 0, all others `depth` below it: what they add is below a
    unit of the large term in fp32 each.  The sum is exactly 1 + n e^-depth;
    every small term is off by the roundings of its exponent (2^-23 of the depth, half of
    that again for the constant), its instruction and its chunk's tree (2.5 * 2^-23); but
    the few in the chunk of the large term are added to it in fp32, half a unit of 1
    for each of three steps.  Results are rounded to fp32."""
    need_gpu()
    x = torch.full((T, V), -float(depth), device="cuda").to(TDT[dtype])
    at = torch.randint(0, V, (T,), device="cuda")
    x[torch.arange(T), at] = 0.0
    rest = (V - 1) * np.exp(-float(depth))
    want = np.log1p(rest)
    tol = rest * 2.0 ** -23 * (1.5 * depth + 2.5) + 3 * 2.0 ** -24 + 2.0 ** -24 * want + 2.0 ** -24 * depth * rest
    assert tol < 0.01 * want or rest < 1e-4
    idx, logp, lse = sg.sg_topk_rows(x, 2)
    check(host(lse), np.full(T, want), tol, "lse of the top rows")
    _, lp, _ = sg.sg_policy_loss(x, at.int(), want_grad=False)
    check(host(lp), np.full(T, -want), tol, "policy")
    off = torch.arange(0, T + 1, device="cuda") if T % 2 == 0 else torch.tensor([0, 1, 2], device="cuda")
    _, S, _ = sg.sg_preference_loss(x, at.int(), off, want_grad=False)
    check(host(S), np.full(S.shape[0], -want), tol, "preference")
    # one listed token that has all the teacher's mass: the loss is -log q
    loss, _ = sg.sg_distill_loss(x, at[:, None].int(), torch.zeros((T, 1), device="cuda"), mode=MODES["plain"])
    check(host(loss), np.full(T, want), tol, "distillation")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(3, 1021), (140, 30011), (2, 70001), (130, 131072)])
def test_distill_at_the_sums_own_bound(T, V, dtype):
    need_gpu()
    x, xs = make_logits(V, T, V, dtype)
    for mode, temp in (("tail", 1.0), ("renorm", 2.0), ("plain", 0.7)):
        idx, logp = make_lists(V, T, V, 20)
        rows = slice(0, 6)
        check_distill(x[rows] if T < 128 else x, idx, logp, mode, dtype, temp, np.linspace(0.5, 1, T))
