"""The vocabulary losses against their definitions in 64 bits: sizes around
the chunk and block limits, odd and strided rows, masks that leave a row
empty, lists with padding, gradients in place, captured into a graph, and on
another stream."""
import numpy as np
import pytest
import torch

import rowloss_ref as ref
import sparse_gradient_synchronization_amd as sg
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

MODES = {"plain": sg.SG_DISTILL_PLAIN, "renorm": sg.SG_DISTILL_RENORM, "tail": sg.SG_DISTILL_TAIL}
KINDS = {"sigmoid": sg.SG_PREF_SIGMOID, "hinge": sg.SG_PREF_HINGE, "ipo": sg.SG_PREF_IPO}
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make_logits(seed, T, V, dtype, ld=None, shift=0, scale=2.0):
    """[T, V] on the GPU inside a buffer of ld columns that starts `shift`
    elements after an aligned address; and the same values as float64."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, V, generator=g) * scale
    hot = torch.randint(0, V, (T, 3), generator=g)
    x.scatter_(1, hot, 3.0 + 6.0 * torch.rand(T, 3, generator=g))
    ld = ld or V
    buf = torch.full((T * ld + shift,), 7.0, dtype=TDT[dtype], device="cuda")
    view = buf[shift:].view(T, ld)[:, :V]
    view.copy_(x.to(TDT[dtype]))
    return view, view.double().cpu().numpy()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def check(got, want, tol, what):
    got, want, tol = np.asarray(got, np.float64), np.asarray(want, np.float64), np.broadcast_to(tol, np.shape(want))
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - want) <= tol)
    bad = np.argwhere(~ok)
    assert bad.size == 0, "%s: %d off, first at %s: got %r want %r tolerance %r" % (
        what, len(bad), bad[0], got[tuple(bad[0])], want[tuple(bad[0])], tol[tuple(bad[0])])


def depth(x, it):
    m = x.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        d = (np.where(np.isfinite(m), m, 0.0) - x) * it
    return np.clip(np.where(np.isfinite(d), d, 0.0), 0, 110)


def host(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------
def make_lists(seed, T, V, k, pad=True):
    """Distinct tokens in random order, masses that sum to less than one, some lists cut short by padding."""
    rng = np.random.default_rng(seed)
    idx = np.empty((T, k), np.int64)
    logp = np.empty((T, k), np.float32)
    for t in range(T):
        idx[t] = rng.choice(V, k, replace=False) if V < 4 * k else np.array(
            sorted(set(rng.integers(0, V, 4 * k)), key=lambda _: rng.random())[:k])
        p = rng.dirichlet(np.full(k, 0.5)) * rng.uniform(0.3, 0.999)
        logp[t] = np.log(np.maximum(p, 1e-12))
        if pad and t % 3 == 1:
            idx[t, rng.integers(0, k + 1):] = (-1, V, 2 ** 31 - 1)[t % 2]
    return idx, logp


def distill_reference(x, idx, logp, w, it, mode):
    T, V = x.shape
    loss, grad, tol_l, tol_g = np.zeros(T), np.zeros((T, V)), np.zeros(T), np.zeros((T, V))
    dep = depth(x, it)
    for t in range(T):
        if w[t] == 0:
            continue
        L, g, scale = ref.distill_row(x[t], idx[t], logp[t].astype(np.float64), it, mode)
        loss[t], grad[t] = w[t] * L, w[t] * g
        # the loss moves with lse (mass at most 1) and, in the tail's term, with the ratio of two sums
        tol_l[t] = abs(w[t]) * 3 * ref.sum_error(V) + 2.0 ** -24 * abs(w[t] * L)
        tol_g[t] = abs(w[t]) * scale * 2 * ref.grad_error(V, dep[t])
    return loss, grad, tol_l, tol_g


def run_distill(x, xs, idx, logp, w, temp, mode, dtype, grad=None):
    loss, g = sg.sg_distill_loss(x, dev(idx, torch.int32), dev(logp, torch.float32), temperature=temp,
                                 mode=MODES[mode], weight=None if w is None else dev(w, torch.float32), grad=grad)
    T, V = xs.shape
    w = np.ones(T) if w is None else w.astype(np.float64)
    L, G, tl, tg = distill_reference(xs, idx, logp, w, 1.0 / temp, mode)
    check(host(loss), L, tl, "loss")
    check(host(g), G, tg + ref.HALF[dtype] * np.abs(G) + 1e-38, "gradient")
    assert sg.sg_device_error() == 0
    return loss, g


# below, at and above a 16-byte chunk, a block of chunks, the rows kept in
# registers and the whole-row limit
SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (3, 255), (7, 1000), (5, 2048), (6, 4099), (3, 16384), (4, 32000),
         (2, 65536), (3, 70001), (2, 131072), (2, 131083), (2, 262144), (1, 262153), (300, 1030), (270, 9001)]
# the same limits with enough rows that none is split over blocks
MANY = [(200, 2048), (200, 2051), (150, 8200), (140, 16390), (130, 33000), (129, 66001)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", SIZES + MANY)
def test_distill_sizes(T, V, dtype):
    need_gpu()
    k = min(V, 1 + (T * 7 + V) % 40)
    mode = ("tail", "renorm", "plain")[(T + V) % 3]
    x, xs = make_logits(T + V, T, V, dtype)
    idx, logp = make_lists(V, T, V, k)
    w = np.linspace(0.5, 1.5, T).astype(np.float32)
    run_distill(x, xs, idx, logp, w, (1.0, 2.0, 0.7)[V % 3], mode, dtype)


@pytest.mark.parametrize("mode", ["tail", "renorm", "plain"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", [1, 63, 64, 65, 700, 1024])
def test_distill_lists(k, mode, dtype):
    need_gpu()
    x, xs = make_logits(k, 5, 5003, dtype)
    idx, logp = make_lists(k + 1, 5, 5003, k)
    run_distill(x, xs, idx, logp, None, 1.0, mode, dtype)


@pytest.mark.parametrize("mode", ["tail", "renorm", "plain"])
def test_distill_whole_vocabulary_and_agreement(mode):
    """The list covers every token (no remainder to share), and a student
    that equals the teacher has loss and gradient near zero."""
    need_gpu()
    T, V = 4, 90
    x, xs = make_logits(3, T, V, "f32")
    idx = np.stack([np.random.default_rng(t).permutation(V) for t in range(T)])
    logp = np.stack([ref.log_softmax(xs[t], 1.0)[0][idx[t]] for t in range(T)]).astype(np.float32)
    loss, g = run_distill(x, xs, idx, logp, None, 1.0, mode, "f32")
    assert host(loss).max() < 1e-4 and np.abs(host(g)).max() < 1e-5


@pytest.mark.parametrize("mode", ["tail", "renorm", "plain"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_empty_rows(mode, dtype):
    """Rows of weight 0 hold NaN; masked tokens (-inf) inside and outside the
    list; a row whose every logit is -inf; a list of padding only."""
    need_gpu()
    T, V, k = 7, 1003, 12
    x, xs = make_logits(5, T, V, dtype)
    idx, logp = make_lists(6, T, V, k, pad=False)
    x[0] = float("nan")
    x[1, ::2] = -float("inf")
    x[1, dev(idx[1], torch.int64)] = 1.0
    x[2] = -float("inf")
    x[3, int(idx[3, 4])] = -float("inf")
    idx[4] = -1
    x[5] = -float("inf")
    x[5, dev(idx[5], torch.int64)] = 2.0
    x[6] = torch.finfo(TDT[dtype]).min
    xs = host(x)
    w = np.ones(T, np.float32)
    w[0] = 0.0
    loss, g = run_distill(x, xs, idx, logp, w, 1.0, mode, dtype)
    assert host(loss)[0] == 0 and not host(g)[0].any()
    assert host(loss)[2] == np.inf and host(loss)[3] == np.inf
    assert host(loss)[4] == 0 or mode == "tail"


def test_distill_nan_stays_in_its_row():
    need_gpu()
    x, xs = make_logits(8, 6, 5000, "f32")
    idx, logp = make_lists(9, 6, 5000, 8, pad=False)
    x[2, 4321] = float("nan")
    x[4, 17] = float("inf")
    loss, g = sg.sg_distill_loss(x, dev(idx, torch.int32), dev(logp, torch.float32))
    bad = ~np.isfinite(host(loss))
    assert list(np.flatnonzero(bad)) == [2, 4]
    assert list(np.flatnonzero(~np.isfinite(host(g)).all(1))) == [2, 4]


def test_distill_repeated_token_is_reported():
    need_gpu()
    x, _ = make_logits(10, 3, 500, "f32")
    idx, logp = make_lists(11, 3, 500, 9, pad=False)
    idx[1, 3] = idx[1, 7]
    sg.sg_distill_loss(x, dev(idx, torch.int32), dev(logp, torch.float32))
    assert sg.sg_device_error() == -7
    assert sg.sg_device_error() == 0


# ---------------------------------------------------------------------------
# policy
# ---------------------------------------------------------------------------
def policy_inputs(seed, xs, it):
    T, V = xs.shape
    rng = np.random.default_rng(seed)
    a = np.where(rng.random(T) < 0.7, xs.argmax(1), rng.integers(0, V, T))
    lp = np.array([ref.log_softmax(xs[t], it)[0][a[t]] for t in range(T)])
    old = (lp + rng.normal(0, 0.25, T)).astype(np.float32)
    rf = (lp + rng.normal(0, 0.4, T)).astype(np.float32)
    return a, old, rf, rng.normal(0, 1, T).astype(np.float32)


def run_policy(x, xs, a, old, rf, adv, w, temp, lo, hi, kl, dtype, grad=None, stream=None):
    f = torch.float32
    d = [None if v is None else dev(v, f) for v in (old, adv, rf, w)]
    loss, logp, g = sg.sg_policy_loss(x, dev(a, torch.int32), d[0], d[1], ref_logp=d[2], weight=d[3], clip_low=lo,
                                      clip_high=hi, kl_coef=kl, temperature=temp, grad=grad)
    T, V = xs.shape
    L, P, G = np.zeros(T), np.zeros(T), np.zeros((T, V))
    tl, tp, tg = np.zeros(T), np.zeros(T), np.zeros((T, V))
    dep, se = depth(xs, 1.0 / temp), ref.sum_error(V)
    for t in range(T):
        wt = 1.0 if w is None else float(w[t])
        if wt == 0 or not 0 <= a[t] < V:
            continue
        o, r_, A = (None if old is None else float(old[t])), (None if rf is None else float(rf[t])), (0.0 if adv is None else float(adv[t]))
        l, p, gr = ref.policy_row(xs[t], a[t], o, r_, A, 1.0 / temp, lo, hi, kl)
        L[t], P[t], G[t] = wt * l, p, wt * gr
        ratio = 1.0 if o is None else np.exp(p - o)
        # the loss's slope in logp times logp's error; the gradient's slope is off by its own derivative times it
        move = abs(ratio * A) + (kl * abs(1 - np.exp(r_ - p)) if r_ is not None else 0.0)
        bend = abs(ratio * A) + (kl * np.exp(r_ - p) if r_ is not None else 0.0)
        tl[t] = abs(wt) * (move + bend * se) * se + 2.0 ** -24 * abs(L[t])
        tp[t] = se + 2.0 ** -24 * abs(p)
        e = np.zeros(V)
        e[a[t]] = 1.0
        q = np.exp(ref.log_softmax(xs[t], 1.0 / temp)[0])
        tg[t] = np.abs(G[t]) * 2 * ref.grad_error(V, dep[t]) + abs(wt) / temp * (bend * np.abs(e - q) + (move + bend) * q) * 2 * se
    check(host(logp), P, tp, "logp")
    check(host(loss), L, tl, "loss")
    if g is not None:
        check(host(g), G, tg + ref.HALF[dtype] * np.abs(G) + 1e-38, "gradient")
    return loss, logp, g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", SIZES + MANY)
def test_policy_sizes(T, V, dtype):
    need_gpu()
    temp = (1.0, 0.7, 2.0)[(T + V) % 3]
    x, xs = make_logits(T * 3 + V, T, V, dtype)
    a, old, rf, adv = policy_inputs(V, xs, 1.0 / temp)
    w = np.linspace(0.2, 1.0, T).astype(np.float32)
    run_policy(x, xs, a, old, rf, adv, w, temp, 0.2, 0.28, 0.05, dtype)


@pytest.mark.parametrize("old,rf,adv,kl", [(False, False, True, 0.0), (True, False, True, 0.1), (False, True, True, 0.1),
                                           (True, True, False, 1.0), (False, False, False, 0.0), (True, True, True, 0.0)])
def test_policy_optional_inputs(old, rf, adv, kl):
    need_gpu()
    x, xs = make_logits(21, 9, 777, "f32")
    a, o, r, A = policy_inputs(22, xs, 1.0)
    run_policy(x, xs, a, o if old else None, r if rf and kl else None, A if adv else None, None, 1.0, 0.1, 0.3, kl, "f32")


def test_policy_clipped_rows_have_no_gradient_without_kl():
    need_gpu()
    T, V = 8, 600
    x, xs = make_logits(23, T, V, "f32")
    a, _, _, _ = policy_inputs(24, xs, 1.0)
    lp = np.array([ref.log_softmax(xs[t], 1.0)[0][a[t]] for t in range(T)])
    old = (lp + np.array([-1, -1, 1, 1, -.05, .05, 0, 0])).astype(np.float32)  # ratios e, e, 1/e, 1/e, near 1
    adv = np.array([1, -1, 1, -1, 1, 1, -1, 0], np.float32)
    _, _, g = run_policy(x, xs, a, old, None, adv, None, 1.0, 0.2, 0.2, 0.0, "f32")
    moved = np.abs(host(g)).max(1) > 0
    assert list(moved) == [False, True, True, False, True, True, True, False]


def test_policy_masks():
    """Weight 0 and actions outside the vocabulary: the row is not read;
    actions on a masked token; a row of nothing; a NaN kept in its row."""
    need_gpu()
    T, V = 8, 1200
    x, xs = make_logits(25, T, V, "bf16")
    a, old, rf, adv = policy_inputs(26, xs, 1.0)
    w = np.ones(T, np.float32)
    x[0], w[0] = float("nan"), 0.0
    x[1], a[1] = float("nan"), -1
    a[2] = V
    x[3, 5:] = -float("inf")
    a[3] = 2
    x[4, int(a[4])] = -float("inf")
    adv[4] = 1.0
    x[5, 100] = float("nan")
    loss, logp, g = sg.sg_policy_loss(x, dev(a, torch.int32), dev(old, torch.float32), dev(adv, torch.float32),
                                      weight=dev(w, torch.float32))
    loss, logp, g = host(loss), host(logp), host(g)
    for t in (0, 1, 2):
        assert loss[t] == 0 and logp[t] == 0 and not g[t].any()
    lq = ref.log_softmax(host(x)[3], 1.0)[0]
    assert abs(logp[3] - lq[2]) < 1e-5 and not g[3, 5:].any()
    assert logp[4] == -np.inf and loss[4] == 0 and not g[4].any()  # ratio 0
    assert np.isnan(loss[5]) and np.isnan(logp[5])
    assert np.isfinite(g[6:]).all() and np.isfinite(loss[6:]).all()


# ---------------------------------------------------------------------------
# preference
# ---------------------------------------------------------------------------
def pref_inputs(seed, xs, B, masked=0.25):
    T, V = xs.shape
    rng = np.random.default_rng(seed)
    off = np.concatenate([[0], np.sort(rng.integers(0, T + 1, 2 * B - 1)), [T]])
    label = rng.integers(0, V, T)
    label[rng.random(T) < masked] = -1
    S = np.zeros(2 * B)
    for s in range(2 * B):
        S[s] = sum(ref.log_softmax(xs[t], 1.0)[0][label[t]] for t in range(off[s], off[s + 1]) if label[t] >= 0)
    return label, off, S, rng


def run_pref(x, xs, label, off, rf, w, kind, beta, eps, average, dtype, grad=None):
    B = (len(off) - 1) // 2
    loss, S, g = sg.sg_preference_loss(x, dev(label, torch.int32), dev(off, torch.int64),
                                       ref_logp=None if rf is None else dev(rf, torch.float32),
                                       weight=None if w is None else dev(w, torch.float32), kind=KINDS[kind],
                                       beta=beta, smoothing=eps, average=average, grad=grad)
    T, V = xs.shape
    rf64 = np.zeros(2 * B) if rf is None else rf.astype(np.float64)
    w64 = np.ones(B) if w is None else w.astype(np.float64)
    L, P, G = ref.preference(xs, label, off, rf64, w64, kind, beta, eps if kind == "sigmoid" else 0.0, average)
    se = ref.sum_error(V)
    n = np.array([sum(0 <= label[t] < V for t in range(off[s], off[s + 1])) for s in range(2 * B)])
    each = np.where(n > 0, 1, 0) if average else n
    derr = (each[:B] + each[B:]) * se  # error of d
    d = (P[:B] - rf64[:B]) - (P[B:] - rf64[B:])
    slope = {"ipo": 2 * np.abs(d - 0.5 / beta), "hinge": np.full(B, beta), "sigmoid": np.full(B, beta)}[kind]
    bend = {"ipo": 2.0, "hinge": 0.0, "sigmoid": beta * beta}[kind]
    check(host(S), P, each * se + 2.0 ** -24 * np.abs(P), "sequence logp")
    check(host(loss), L, np.abs(w64) * (slope + bend * derr) * derr + 2.0 ** -24 * np.abs(L), "loss")
    if g is not None:
        tol = np.abs(G) * (2 * ref.grad_error(V, depth(xs, 1.0)) + ref.HALF[dtype]) + 1e-38
        for s in range(2 * B):
            per = 1.0 / max(1, n[s]) if average else 1.0
            for t in range(off[s], off[s + 1]):
                if 0 <= label[t] < V:
                    q = np.exp(ref.log_softmax(xs[t], 1.0)[0])
                    e = np.zeros(V)
                    e[label[t]] = 1.0
                    b = s % B
                    # the slope's own error, and 1 - q of the label at the sum's error
                    tol[t] += abs(w64[b]) * per * (bend * derr[b] * np.abs(e - q) + slope[b] * q * 2 * se)
        check(host(g), G, tol, "gradient")
    return loss, S, g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [s for s in SIZES if s[0] * s[1] < 700000])
def test_preference_sizes(T, V, dtype):
    need_gpu()
    x, xs = make_logits(T * 5 + V, T, V, dtype)
    B = max(1, T // 6)
    label, off, S, rng = pref_inputs(V, xs, B)
    rf = (S + rng.normal(0, 1, 2 * B)).astype(np.float32)
    kind = ("sigmoid", "ipo", "hinge")[(T + V) % 3]
    run_pref(x, xs, label, off, rf, np.linspace(0.5, 1, B).astype(np.float32), kind, 0.3, 0.1, False, dtype)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("reference", [False, True])
def test_preference_kinds(kind, average, reference):
    need_gpu()
    x, xs = make_logits(31, 40, 500, "f32")
    label, off, S, rng = pref_inputs(32, xs, 5)
    off[3] = off[4]  # an empty sequence
    rf = rng.normal(0, 1, 10).astype(np.float32) if reference else None
    run_pref(x, xs, label, off, rf, None, kind, 0.2, 0.05 if kind == "sigmoid" else 0.0, average, "f32")


def test_preference_rows_that_do_not_count():
    """Rows of no sequence and rows without a label are not read; a pair of weight 0."""
    need_gpu()
    T, V = 30, 900
    x, xs = make_logits(33, T, V, "bf16")
    off = np.array([4, 10, 16, 22, 27])
    label = np.random.default_rng(34).integers(0, V, T)
    label[[5, 17]] = (-100, V)
    outside = [0, 1, 2, 3, 27, 28, 29]
    x[5], x[17] = float("nan"), float("inf")
    keep = x.clone()
    x[outside] = float("nan")
    xs = host(keep)
    xs[[5, 17]] = 0.0
    w = np.array([1.0, 0.0], np.float32)
    loss, S, g = sg.sg_preference_loss(x, dev(label, torch.int32), dev(off, torch.int64), weight=dev(w, torch.float32))
    L, P, G = ref.preference(xs, label, off, np.zeros(4), w.astype(np.float64), "sigmoid", 0.1, 0.0, False)
    check(host(S), P, 6 * ref.sum_error(V) + 2.0 ** -24 * np.abs(P), "sequence logp")
    g = host(g)
    assert not g[outside].any() and not g[5].any() and not g[17].any() and host(loss)[1] == 0
    assert not g[10:16].any() and not g[22:27].any()  # pair 1 has weight 0
    assert np.abs(g[4]).max() > 0 and np.abs(g[18]).max() > 0


def test_preference_no_rows_and_bad_offsets():
    need_gpu()
    x = torch.zeros(0, 50, device="cuda")
    loss, S, g = sg.sg_preference_loss(x, dev(np.zeros(0), torch.int32), dev(np.zeros(5), torch.int64))
    check(host(loss), np.full(2, np.log(2.0)), 1e-7, "empty pairs")
    assert g.shape == (0, 50) and sg.sg_device_error() == 0
    x, xs = make_logits(35, 6, 100, "f32")
    label = np.arange(6)
    for off in ([0, 4, 2, 5, 6], [0, 2, 3, 5, 9]):
        sg.sg_preference_loss(x, dev(label, torch.int32), dev(np.array(off), torch.int64))
        assert sg.sg_device_error() == -7
    assert sg.sg_device_error() == 0


# ---------------------------------------------------------------------------
# layouts, streams, graphs
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,ld,shift", [(1000, 1024, 0), (1001, 1001, 1), (1001, 1007, 3), (9000, 9001, 5),
                                        (70000, 70003, 1), (131072, 131079, 7)])
def test_strided_and_unaligned_rows(V, ld, shift, dtype):
    """Padded and unaligned logits, a gradient with a stride of its own whose
    padding stays untouched, and the same call in place."""
    need_gpu()
    T = 4
    x, xs = make_logits(V + ld, T, V, dtype, ld, shift)
    a, old, rf, adv = policy_inputs(41, xs, 1.0)
    buf = torch.full((T, V + 11), 5.0, dtype=TDT[dtype], device="cuda")
    _, _, g = run_policy(x, xs, a, old, rf, adv, None, 1.0, 0.2, 0.2, 0.1, dtype, grad=buf[:, :V])
    assert (buf[:, V:] == 5.0).all()
    base = x._base if x._base is not None else x
    before = base.clone()
    _, _, same = run_policy(x, xs, a, old, rf, adv, None, 1.0, 0.2, 0.2, 0.1, dtype, grad=x)
    assert same.data_ptr() == x.data_ptr()
    assert torch.equal(same, g)
    inside = torch.zeros(base.numel(), dtype=torch.bool, device="cuda")
    inside[shift:].view(T, ld)[:, :V] = True
    assert torch.equal(base.view(-1)[~inside], before.view(-1)[~inside])


@pytest.mark.parametrize("T,V", [(3, 40000), (300, 5000), (2, 140001), (280, 66000)])
def test_in_place_equals_out_of_place(T, V):
    need_gpu()
    x, _ = make_logits(50, T, V, "bf16")
    idx, logp = make_lists(51, T, V, 20)
    idx, logp = dev(idx, torch.int32), dev(logp, torch.float32)
    loss, g = sg.sg_distill_loss(x, idx, logp)
    label = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    off = torch.tensor([0, T // 2, T], device="cuda")
    off = torch.cat([off[:2], off[2:]])
    lp, sp, gp = sg.sg_preference_loss(x, label, off[[0, 1, 2]])
    y = x.clone()
    loss2, g2 = sg.sg_distill_loss(y, idx, logp, grad=y)
    assert torch.equal(loss, loss2) and torch.equal(g, g2) and g2.data_ptr() == y.data_ptr()
    y = x.clone()
    lp2, sp2, gp2 = sg.sg_preference_loss(y, label, off[[0, 1, 2]], grad=y)
    assert torch.equal(lp, lp2) and torch.equal(sp, sp2) and torch.equal(gp, gp2)


def test_loss_without_gradient_is_the_same():
    need_gpu()
    for T, V in ((5, 3001), (300, 2100), (4, 150000)):
        x, xs = make_logits(60, T, V, "bf16")
        idx, logp = make_lists(61, T, V, 16)
        idx, logp = dev(idx, torch.int32), dev(logp, torch.float32)
        a, _ = sg.sg_distill_loss(x, idx, logp)
        b, none = sg.sg_distill_loss(x, idx, logp, want_grad=False)
        assert none is None
        check(host(b), host(a), 2 * 3 * ref.sum_error(V) + 2.0 ** -23 * np.abs(host(a)), "loss alone")


def test_offsets_beyond_32_bits():
    """More than 2^32 elements: the last rows give what they give alone."""
    need_gpu()
    T, V = 33000, 131080
    x = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    tail, xs = make_logits(70, 3, V, "bf16")
    x[-3:] = tail
    a, old, rf, adv = policy_inputs(71, xs, 1.0)
    w = torch.zeros(T, device="cuda")
    w[-3:] = 1.0
    full = lambda v, dt: torch.cat([torch.zeros(T - 3, dtype=dt, device="cuda"), dev(v, dt)])  # noqa: E731
    f = torch.float32
    loss, logp, g = sg.sg_policy_loss(x, full(a, torch.int32), full(old, f), full(adv, f), weight=w, grad=x)
    loss3, logp3, g3 = sg.sg_policy_loss(tail, dev(a, torch.int32), dev(old, f), dev(adv, f))
    tol = 4 * ref.sum_error(V)
    check(host(loss[-3:]), host(loss3), tol * (1 + np.abs(host(loss3))), "loss")
    check(host(logp[-3:]), host(logp3), tol * (1 + np.abs(host(logp3))), "logp")
    check(host(g[-3:]), host(g3), 2 * ref.HALF["bf16"] * np.abs(host(g3)) + tol, "gradient")
    assert not loss[:-3].any() and not g[:-3].any()
    idx = torch.full((T, 4), -1, dtype=torch.int32, device="cuda")
    idx[-1] = torch.tensor([5, 9, V - 1, 70000], dtype=torch.int32)
    x[-3:] = tail
    lp = torch.full((T, 4), -2.0, device="cuda")
    w[:-1] = 0.0
    loss, _ = sg.sg_distill_loss(x, idx, lp, weight=w, want_grad=False)
    loss1, _ = sg.sg_distill_loss(tail[2:], idx[-1:], lp[-1:], want_grad=False)
    check(host(loss[-1:]), host(loss1), tol * (1 + np.abs(host(loss1))), "distill")


def test_many_rows_longer_than_a_bitmap():
    """Lists over rows of more than 2^18 tokens, in parts whatever the number of rows."""
    need_gpu()
    T, V, k = 130, 262200, 9
    x = torch.randn((T, V), device="cuda").bfloat16()
    idx, logp = make_lists(72, T, V, k)
    idx, logp = dev(idx, torch.int32), dev(logp, torch.float32)
    loss, g = sg.sg_distill_loss(x, idx, logp)
    for r in (0, 64, 127):
        loss3, g3 = sg.sg_distill_loss(x[r:r + 3], idx[r:r + 3], logp[r:r + 3])
        L, G, tl, tg = distill_reference(host(x[r:r + 1]), idx[r:r + 1].cpu().numpy(), logp[r:r + 1].cpu().numpy(),
                                         np.ones(1), 1.0, "tail")
        for a, b in ((loss[r:r + 1], g[r:r + 1]), (loss3[:1], g3[:1])):
            check(host(a), L, tl, "loss")
            check(host(b), G, tg + ref.HALF["bf16"] * np.abs(G) + 1e-38, "gradient")


def test_split_rows_beyond_a_grid_dimension():
    """65540 rows in parts: the last ones are those of a short call."""
    need_gpu()
    T, V = 65540, 262200
    x = torch.empty((T, V), dtype=torch.bfloat16, device="cuda")  # rows of weight 0 are not read
    tail, _ = make_logits(73, 3, V, "bf16")
    x[-3:] = tail
    idx = torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
    idx[-3:] = torch.tensor([7, V - 2], dtype=torch.int32)
    lp = torch.full((T, 2), -1.5, device="cuda")
    w = torch.zeros(T, device="cuda")
    w[-3:] = 1.0
    loss, _ = sg.sg_distill_loss(x, idx, lp, weight=w, want_grad=False)
    loss3, _ = sg.sg_distill_loss(tail, idx[-3:], lp[-3:], want_grad=False)
    check(host(loss[-3:]), host(loss3), 8 * ref.sum_error(V), "loss")
    assert not loss[:-3].any()


@pytest.mark.parametrize("V", [33000, 140001])
def test_on_another_stream_and_in_a_graph(V):
    """Queued on a side stream; captured once and replayed with new inputs,
    eager work between the replays.  The longer rows are split."""
    need_gpu()
    T, k = 12, 16
    x, _ = make_logits(80, T, V, "bf16")
    idx, logp = make_lists(81, T, V, k)
    idx, logp = dev(idx, torch.int32), dev(logp, torch.float32)
    a = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    adv = torch.randn(T, device="cuda")
    off = torch.tensor([0, 5, T], device="cuda")

    def step():
        return (sg.sg_distill_loss(x, idx, logp) + sg.sg_policy_loss(x, a, None, adv)
                + sg.sg_preference_loss(x, a, off) + sg.sg_topk_rows(x, k))

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    for p, q in zip(other, eager):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(3):
        y, _ = make_logits(90 + rep, T, V, "bf16")
        x.copy_(y)
        adv.copy_(torch.randn(T, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for p, q in zip(got, step()):
            assert torch.equal(p, q)


def test_results_repeat():
    need_gpu()
    for T, V in ((3, 100000), (400, 20000)):
        x, _ = make_logits(95, T, V, "bf16")
        idx, logp = make_lists(96, T, V, 30)
        idx, logp = dev(idx, torch.int32), dev(logp, torch.float32)
        first = sg.sg_distill_loss(x, idx, logp)
        for _ in range(3):
            again = sg.sg_distill_loss(x, idx, logp)
            assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_long_sequences_keep_their_differences():
    """One pair of thousands of tokens: the sequences' sums are differences of
    thousands, so what every token is off by must not be of one sign."""
    need_gpu()
    T, V = 6000, 1500
    x, xs = make_logits(97, T, V, "f32")
    label = np.random.default_rng(98).integers(0, V, T)
    off = np.array([0, 1000, T])
    lq = np.array([ref.log_softmax(xs[t], 1.0)[0][label[t]] for t in range(T)])
    S = np.array([lq[:1000].sum(), lq[1000:].sum()])
    rf = (S - np.array([3.0, -2.0])).astype(np.float32)
    loss, got, g = sg.sg_preference_loss(x, dev(label, torch.int32), dev(off, torch.int64),
                                         ref_logp=dev(rf, torch.float32), kind=sg.SG_PREF_IPO, beta=0.1)
    d = (S[0] - float(rf[0])) - (S[1] - float(rf[1]))
    want = (d - 5.0) ** 2
    # a token's log-probability is off by a random 1e-7 (an exponential's 2^-23, one sign or the other) and by 1e-8
    # of one sign: 8e-6 + 6e-5 for 6000 of them, and the loss moves by 2 |d - 5| times that
    off_by = np.sqrt(T) * 1e-7 + T * 1e-8
    assert abs(float(loss[0]) - want) <= 2 * abs(d - 5.0) * off_by + off_by ** 2 + 2.0 ** -24 * want


# ---------------------------------------------------------------------------
# gradients against differences of the 64-bit loss
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("what", ["plain", "renorm", "tail", "policy", "sigmoid", "hinge", "ipo"])
def test_gradient_against_differences(what):
    """Central differences of the loss in 64 bits: h = 1e-4 leaves h^2 / 6
    times a third derivative of order one (below 1e-8) and 1e-16 / h of
    rounding (1e-12 of a loss of order one, 1e-10 of an IPO loss of 100); the
    kernel's own error is that of its type."""
    need_gpu()
    T, V, h = 6, 40, 1e-4
    x, xs = make_logits(100, T, V, "f32", scale=1.0)
    if what in MODES:
        idx, logp = make_lists(101, T, V, 7, pad=False)
        _, g = sg.sg_distill_loss(x, dev(idx, torch.int32), dev(logp, torch.float32), temperature=2.0, mode=MODES[what])
        f = lambda y: sum(ref.distill_row(y[t], idx[t], logp[t].astype(np.float64), 0.5, what)[0] for t in range(T))  # noqa: E731
    elif what == "policy":
        a, old, rf, adv = policy_inputs(102, xs, 1.0)
        _, _, g = sg.sg_policy_loss(x, dev(a, torch.int32), dev(old, torch.float32), dev(adv, torch.float32),
                                    ref_logp=dev(rf, torch.float32), kl_coef=0.3)
        f = lambda y: sum(ref.policy_row(y[t], a[t], float(old[t]), float(rf[t]), float(adv[t]), 1.0, 0.2, 0.2, 0.3)[0]  # noqa: E731
                          for t in range(T))
    else:
        label, off, S, _ = pref_inputs(103, xs, 1, masked=0.0)
        off = np.array([0, 3, T])
        label = np.abs(label)
        _, _, g = sg.sg_preference_loss(x, dev(label, torch.int32), dev(off, torch.int64), kind=KINDS[what], beta=0.1,
                                        smoothing=0.1 if what == "sigmoid" else 0.0)
        f = lambda y: ref.preference(y, label, off, np.zeros(2), np.ones(1), what, 0.1, 0.1 if what == "sigmoid" else 0.0, False)[0].sum()  # noqa: E731
    g = host(g)
    scale = max(1.0, np.abs(g).max())
    for t in range(T):
        for i in range(0, V, 3):
            up, down = xs.copy(), xs.copy()
            up[t, i] += h
            down[t, i] -= h
            want = (f(up) - f(down)) / (2 * h)
            assert abs(g[t, i] - want) <= 1e-6 * scale + 4 * ref.sum_error(V) * scale, (t, i, g[t, i], want)
