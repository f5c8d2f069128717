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


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------
MODES = {"plain": sg.SG_DISTILL_PLAIN, "renorm": sg.SG_DISTILL_RENORM, "tail": sg.SG_DISTILL_TAIL}


def sum_bound(V):
    """Bound of the relative error of a row's sum of exponentials, as the
    kernels add it.  A term's exponent is rounded twice (the difference to the
    maximum, its product with the scale): 2^-23 of the term's depth, and the
    depth weighted by the terms' shares is at most log V; the instruction is
    off by 2^-23, the tree of a chunk adds three half units.  All else is added in
    fp64, but where a lane's maximum rises its sum is scaled by an fp32
    exponential: 2^-23 each time (of n chunks in random order that is log n + 1
    times on average; 16 here), and 2^-23 of the rises, which add up to the
    maximum's depth again.  Waves, blocks and parts join with one such scaling each."""
    return 2.0 ** -23 * (2 * max(1.0, np.log(V)) + 1 + 1.5 + 16 + 3)


def distill_bounds(x, idx, logp, w, it, mode):
    """Loss and gradient of the definition, and what the kernel's may be off
    by: the sums' errors; scalars take the temperature as fp32 rounds it, half a
    unit of the distances they multiply; a gradient's factors, exponential and
    product are rounded once each, and its exponent by 3 half units of its own depth
    below the maximum of the listed or of the unlisted tokens."""
    T, V = x.shape
    se = sum_bound(V)
    L, G, tl, tg = np.zeros(T), np.zeros((T, V)), np.zeros(T), np.zeros((T, V))
    for t in range(T):
        l, g, scale = ref.distill_row(x[t], idx[t], logp[t].astype(np.float64), it, mode)
        ok = (idx[t] >= 0) & (idx[t] < V)
        listed = np.zeros(V, bool)
        listed[idx[t][ok]] = True
        depth = np.zeros(V)
        for part, top in ((listed, x[t].max()), (~listed, x[t][~listed].max() if (~listed).any() else 0.0)):
            with np.errstate(invalid="ignore"):
                d = (top - x[t][part]) * it
            depth[part] = np.where(np.isfinite(d), d, 0.0)
        finite = x[t][np.isfinite(x[t])]
        apart = (finite.max() - finite.min()) * it if finite.size else 0.0
        L[t], G[t] = w[t] * l, w[t] * g
        tl[t] = abs(w[t]) * (3 * se + 2.0 ** -24 * 2 * apart) + 2.0 ** -24 * abs(w[t] * l)
        tg[t] = abs(w[t]) * scale * (2 * se + 2.0 ** -22 + 3 * 2.0 ** -24 * np.minimum(depth, 110))
    return L, G, tl, tg


def check_distill(x, idx, logp, mode, dtype, temp=1.0, weight=None):
    T = x.shape[0]
    w = np.ones(T) if weight is None else np.asarray(weight, np.float64)
    args = (dev(idx, torch.int32), dev(logp, torch.float32))
    kw = dict(temperature=temp, mode=MODES[mode], weight=None if weight is None else dev(weight, torch.float32))
    loss, g = sg.sg_distill_loss(x, *args, **kw)
    L, G, tl, tg = distill_bounds(host(x), idx, logp, w, 1.0 / temp, mode)
    check(host(loss), L, tl, "loss")
    # what an exponential below 2^-126 gives is lost
    check(host(g), G, tg + ref.HALF[dtype] * np.abs(G) + 2.0 ** -126 * 16, "gradient")
    alone, _ = sg.sg_distill_loss(x, *args, want_grad=False, **kw)
    check(host(alone), L, tl, "loss without the gradient")
    assert sg.sg_device_error() == 0
    return host(loss), host(g)


# in one block (rows kept in registers, and longer ones) and in parts
GAP_ROWS = [(3, 100), (3, 1000), (3, 5003), (130, 33000), (2, 70001), (1, 262200)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", GAP_ROWS)
@pytest.mark.parametrize("gap,temp", [(80, 1.0), (87, 1.0), (88, 1.0), (95, 1.0), (120, 2.0), (200, 1.0), (600, 1.0),
                                      (60, 0.1)])
def test_tail_gradient_far_below_the_list(gap, temp, T, V, dtype):
    """The unlisted tokens share R however far below the listed ones they lie:
    each of them has a gradient of R times its share among them."""
    need_gpu()
    rng = np.random.default_rng(gap + V)
    g = torch.Generator().manual_seed(gap + V)
    x = (torch.rand((T, V), generator=g) * 0.5 - gap).to(TDT[dtype])
    idx = np.stack([rng.choice(V, 5, replace=False) for _ in range(T)])
    x[torch.arange(T)[:, None], torch.from_numpy(idx)] = torch.randn((T, 5), generator=g).to(TDT[dtype])
    logp = np.log(np.full((T, 5), 0.16)).astype(np.float32)
    _, grad = check_distill(x.cuda(), idx, logp, "tail", dtype, temp)
    listed = np.zeros((T, V), bool)
    np.put_along_axis(listed, idx, True, 1)
    assert np.isfinite(grad).all() and (grad[~listed] < 0).all()
    unlisted = np.where(listed, 0.0, grad).sum(1) * temp
    # R = 0.2 less what q of them adds (e^-80 and less), each rounded to the type
    assert np.abs(unlisted + 0.2).max() < 0.2 * (ref.HALF[dtype] + 2.0 ** -17)


@pytest.mark.parametrize("mode", ["plain", "renorm", "tail"])
@pytest.mark.parametrize("T,V", [(2, 700), (2, 70001)])
def test_distill_listed_far_below_the_others(T, V, mode):
    """The other way round: a list that the student gives no weight to."""
    need_gpu()
    rng = np.random.default_rng(V)
    for gap in (50, 95, 300):
        x = torch.randn((T, V), generator=torch.Generator().manual_seed(gap))
        idx = np.stack([rng.choice(V, 6, replace=False) for _ in range(T)])
        x[torch.arange(T)[:, None], torch.from_numpy(idx)] -= gap
        logp = np.log(rng.dirichlet(np.ones(6), T) * 0.7).astype(np.float32)
        check_distill(x.cuda(), idx, logp, mode, "f32")


@pytest.mark.parametrize("T,V", [(4, 900), (130, 33000), (2, 70001)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("level", [-3, -60, -90, -100, -104, -300, -700, -5000])
def test_renormalised_lists_of_little_mass(level, T, V, dtype):
    """p / P does not depend on the level of the list's log-probabilities:
    the definition is taken from the list lifted to 0, where its sums are ordinary."""
    need_gpu()
    rng = np.random.default_rng(V - level)
    x, xs = make_logits(V - level, T, V, dtype)
    idx = np.stack([rng.choice(V, 70, replace=False) for _ in range(T)])
    idx[::3, 40:] = -1
    logp = (level + rng.normal(0, 1.0, (T, 70))).astype(np.float32)
    logp[1::3, 5] = -np.inf
    loss, g = sg.sg_distill_loss(x, dev(idx, torch.int32), dev(logp, torch.float32), mode=sg.SG_DISTILL_RENORM)
    lifted = logp.astype(np.float64) - level
    L, G, tl, tg = np.zeros(T), np.zeros((T, V)), np.zeros(T), np.zeros((T, V))
    for t in range(T):
        a = distill_bounds(xs[t:t + 1], idx[t:t + 1], lifted[t:t + 1], np.ones(1), 1.0, "renorm")
        L[t], G[t], tl[t], tg[t] = a[0][0], a[1][0], a[2][0], a[3][0]
    check(host(loss), L, tl, "loss")
    check(host(g), G, tg + ref.HALF[dtype] * np.abs(G) + 2.0 ** -126 * 16, "gradient")
    y = x.clone()
    loss2, g2 = sg.sg_distill_loss(y, dev(idx, torch.int32), dev(logp, torch.float32), mode=sg.SG_DISTILL_RENORM, grad=y)
    assert torch.equal(loss, loss2) and torch.equal(g, g2)


@pytest.mark.parametrize("T,V", [(3, 900), (2, 70001)])
def test_renormalised_list_without_mass(T, V):
    need_gpu()
    x, _ = make_logits(V, T, V, "f32")
    idx = np.stack([np.arange(8) for _ in range(T)])
    idx[0] = -1
    logp = np.full((T, 8), -np.inf, np.float32)
    loss, g = sg.sg_distill_loss(x, dev(idx, torch.int32), dev(logp, torch.float32), mode=sg.SG_DISTILL_RENORM)
    assert not loss.any() and not g.any()


# ---------------------------------------------------------------------------
# rows that hold a NaN or +inf
# ---------------------------------------------------------------------------
def poison(x, t, kind, keep=()):
    """Row t gets a NaN or +inf; 'only': NaN beside nothing but -inf.  The tokens of `keep` become -inf."""
    keep = list(keep)
    if kind == "only":
        x[t] = -float("inf")
    x[t, keep] = -float("inf")
    at = next(i for i in range(x.shape[1] - 3, -1, -1) if i not in keep)
    x[t, at] = float("inf") if kind == "inf" else float("nan")


NAN_ROWS = [(4, 60), (4, 5003), (130, 33000), (3, 70001)]


@pytest.mark.parametrize("mode", ["plain", "renorm", "tail"])
@pytest.mark.parametrize("kind", ["nan", "inf", "only"])
@pytest.mark.parametrize("T,V", NAN_ROWS)
def test_distill_rows_with_a_nan(T, V, kind, mode):
    """NaN results, whatever the list: tokens that are -inf, of no mass, or padding only."""
    need_gpu()
    rng = np.random.default_rng(V)
    x, xs = make_logits(V, T, V, "f32")
    idx = np.stack([rng.choice(V, 6, replace=False) for _ in range(T)])
    logp = np.log(rng.dirichlet(np.ones(6), T) * 0.8).astype(np.float32)
    poison(x, 0, kind, idx[0])
    idx[1] = -1
    poison(x, 1, kind)
    logp[2] = -np.inf
    poison(x, 2, kind, idx[2])
    for want_grad in (True, False):
        loss, g = sg.sg_distill_loss(x, dev(idx, torch.int32), dev(logp, torch.float32), mode=MODES[mode],
                                     want_grad=want_grad)
        assert list(np.flatnonzero(np.isnan(host(loss)))) == [0, 1, 2]
        if want_grad:
            assert np.isnan(host(g)[:3]).all() and np.isfinite(host(g)[3:]).all()


@pytest.mark.parametrize("kind", ["nan", "inf", "only"])
@pytest.mark.parametrize("T,V", NAN_ROWS)
def test_policy_rows_with_a_nan(T, V, kind):
    """An action of -inf, and a policy that is its own old one: NaN all the same."""
    need_gpu()
    x, xs = make_logits(V + 1, T, V, "bf16")
    action = np.arange(T) % V
    poison(x, 0, kind, [0])
    poison(x, 1, kind)
    adv = dev(np.linspace(-1, 1, T), torch.float32)
    some = dev(np.full(T, -3.0), torch.float32)
    for old, rf, kl in ((None, None, 0.0), (some, None, 0.0), (None, some, 0.1), (some, some, 0.1)):
        for want_grad in (True, False):
            loss, logp, g = sg.sg_policy_loss(x, dev(action, torch.int32), old, adv, ref_logp=rf, kl_coef=kl,
                                              want_grad=want_grad)
            assert list(np.flatnonzero(np.isnan(host(loss)))) == [0, 1]
            assert list(np.flatnonzero(np.isnan(host(logp)))) == [0, 1]
            if want_grad:
                g = host(g)
                assert np.isnan(g[:2]).all() and np.isfinite(g[2:]).all()


@pytest.mark.parametrize("kind", ["nan", "inf", "only"])
@pytest.mark.parametrize("T,V", NAN_ROWS)
def test_preference_rows_with_a_nan(T, V, kind):
    """A label of -inf in a row with a NaN: the sequence's sum is NaN, not -inf."""
    need_gpu()
    x, xs = make_logits(V + 2, T, V, "f32")
    label = np.arange(T) % V
    poison(x, 1, kind, [1])
    off = np.array([0, 1, 2, T, T])  # the chosen: row 0, row 1; the rejected: the others, none
    loss, S, g = sg.sg_preference_loss(x, dev(label, torch.int32), dev(off, torch.int64))
    assert list(np.isnan(host(loss))) == [False, True]
    assert list(np.isnan(host(S))) == [False, True, False, False]
    assert np.isnan(host(g)[1]).all() and np.isfinite(np.delete(host(g), 1, 0)).all()


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("T,V", [(6, 700), (1100, 700), (6, 70001)])
def test_a_nan_reaches_its_whole_pair(T, V, kind):
    """And no other: both sequences' gradients, in every kind of loss."""
    need_gpu()
    x, xs = make_logits(V + 3, T, V, "f32")
    label = np.arange(T) % V
    label[3] = -1
    x[1, V - 1] = float("nan")
    off = np.array([0, 2, 3, 5, T])  # rows 0, 1 against 3, 4; row 2 against the rest
    loss, S, g = sg.sg_preference_loss(x, dev(label, torch.int32), dev(off, torch.int64),
                                       kind={"sigmoid": 0, "hinge": 1, "ipo": 2}[kind])
    assert list(np.isnan(host(loss))) == [True, False]
    assert list(np.isnan(host(S))) == [True, False, False, False]
    g = host(g)
    assert np.isnan(g[[0, 1, 4]]).all() and not g[3].any() and np.isfinite(g[2]).all() and np.isfinite(g[5:]).all()


@pytest.mark.parametrize("kind", ["nan", "inf", "only"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", NAN_ROWS)
def test_top_rows_with_a_nan(T, V, dtype, kind):
    """Every log-probability of the row is NaN, those of listed -inf too."""
    need_gpu()
    x, xs = make_logits(V + 4, T, V, dtype)
    k = 12
    poison(x, 1, kind, range(V - 2 - k, V - 3))
    x[1, :V - 2 - k] = -float("inf")  # so that -inf is among the k
    x[1, V - 2:] = -float("inf")
    x[2] = -float("inf")
    idx, logp, lse = sg.sg_topk_rows(x, k)
    assert list(np.flatnonzero(np.isnan(host(lse)))) == [1]
    logp = host(logp)
    assert np.isnan(logp[1]).all() and (logp[2] == -np.inf).all() and np.isfinite(np.delete(logp, [1, 2], 0)).all()
    assert idx[2].tolist() == list(range(k)) and idx[1].tolist() == list(range(k - 1)) + [V - 3]


# ---------------------------------------------------------------------------
# policy
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,V", [(4, 300), (130, 33000), (3, 70001)])
def test_kl_of_an_action_of_probability_zero(T, V):
    """exp(d) - d - 1 goes to +inf with d = ref - logp; the other rows keep theirs."""
    need_gpu()
    x, xs = make_logits(V + 5, T, V, "f32")
    action = np.arange(T) % V
    rf = np.full(T, -2.0, np.float32)
    kw = dict(old_logp=dev(rf, torch.float32), ref_logp=dev(rf, torch.float32), adv=dev(np.ones(T), torch.float32), kl_coef=0.1)
    want, _, _ = sg.sg_policy_loss(x, dev(action, torch.int32), **kw)
    x[1, 1] = -float("inf")
    x[2] = -float("inf")
    for want_grad in (True, False):
        loss, logp, g = sg.sg_policy_loss(x, dev(action, torch.int32), want_grad=want_grad, **kw)
        assert (host(loss)[1:3] == np.inf).all() and (host(logp)[1:3] == -np.inf).all()
        # without the gradient other threads add a row's terms
        check(np.delete(host(loss), [1, 2]), np.delete(host(want), [1, 2]),
              2 * sum_bound(V) * 2 * (1 + np.abs(np.delete(host(want), [1, 2]))), "the others' loss")
        if want_grad:
            assert not np.isfinite(host(g)[1, 1]) and np.isfinite(np.delete(host(g), [1, 2], 0)).all()


# ---------------------------------------------------------------------------
# temperatures
# ---------------------------------------------------------------------------
def test_highest_temperatures():
    """A uniform distribution over what is not masked, up to the limit; beyond it the call is refused."""
    need_gpu()
    x, xs = make_logits(7, 3, 1000, "f32")
    x[:, ::2] = -float("inf")
    action = torch.tensor([1, 3, 4], device="cuda", dtype=torch.int32)
    uniform = -np.log(500.0)
    for temp in (1e20, 1e30, 1e37):
        idx, logp, lse = sg.sg_topk_rows(x, 500, temperature=temp)
        check(host(logp), np.full((3, 500), uniform), sum_bound(1000) + 2.0 ** -24 * abs(uniform), "logp")
        loss, logp, g = sg.sg_policy_loss(x, action, None, torch.ones(3, device="cuda"), temperature=temp)
        check(host(logp), [uniform, uniform, -np.inf], sum_bound(1000) + 2.0 ** -24 * abs(uniform), "logp")
        assert torch.isfinite(g).all()
    for temp in (1.2e37, 1e39, 1e300):
        with pytest.raises(sg.SgError):
            sg.sg_topk_rows(x, 5, temperature=temp)
