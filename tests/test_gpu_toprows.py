"""The rows' top logits against a stable sort in 64 bits: indices equal,
ties to the lowest index, log-probabilities within the sum's error."""
import numpy as np
import pytest
import torch

import rowloss_ref as ref
import sparse_gradient_synchronization_amd as sg
from gpu_util import need_gpu
from test_gpu_rowloss import MANY, SIZES, TDT, check, host, make_logits

pytestmark = pytest.mark.gpu


def run(x, xs, k, temp=1.0):
    idx, logp, lse = sg.sg_topk_rows(x, k, temperature=temp)
    ri, rp, rl = ref.topk_rows(xs, k, 1.0 / temp)
    se = ref.sum_error(xs.shape[1])
    assert np.array_equal(idx.cpu().numpy().view(np.uint32), ri)
    check(host(lse), rl, se + 2.0 ** -24 * np.abs(rl), "lse")
    check(host(logp), rp, se + 2.0 ** -24 * np.abs(rp), "logp")
    assert sg.sg_device_error() == 0
    return idx, logp, lse


# the longest row of a wave and the next one, the longest whose line maxima fit
# (one line more takes the whole-row select), with and without parts
EDGES = [(3, 4095), (3, 4096), (3, 4097), (130, 4096), (130, 2048), (130, 2049), (1, 300001), (1, 1 << 20),
         (129, 262144), (129, 262145), (2, 524287), (2, 524288)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", SIZES + MANY + EDGES)
def test_sizes(T, V, dtype):
    need_gpu()
    x, xs = make_logits(T + 2 * V, T, V, dtype)
    for k in sorted({1, min(V, 1 + (V * 3 + T) % 60), min(V, 256)}):
        if T * V < 10000000 or k > 1:
            run(x, xs, k, (1.0, 2.0, 0.7)[V % 3])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2, 300])
@pytest.mark.parametrize("k", [1, 2, 63, 64, 65, 511, 512, 513, 1023, 1024])
def test_list_lengths(k, T, dtype):
    need_gpu()
    for V in (1100, 4001, 9001) if T > 2 else (1100, 4001, 9001, 140001):
        x, xs = make_logits(k, T, V, dtype)
        run(x, xs, k)


@pytest.mark.parametrize("T", [1, 260])
@pytest.mark.parametrize("V", [40, 3000, 20000, 66000])
@pytest.mark.parametrize("kind", ["equal", "two", "ascending", "descending", "clustered", "one_lane", "masked",
                                  "zeros", "lowest"])
def test_orders_and_ties(V, T, kind):
    """Ties everywhere, sorted rows, all large values side by side or far
    apart at one lane's places, rows with fewer finite logits than k."""
    need_gpu()
    T = T if V <= 3000 else min(T, 3)
    rng = np.random.default_rng(V)
    rows = []
    for t in range(T):
        if kind == "equal":
            v = np.full(V, 1.5)
        elif kind == "two":
            v = rng.integers(0, 2, V) * 2.0 - 1.0
        elif kind == "ascending":
            v = np.linspace(-4, 4, V)
        elif kind == "descending":
            v = np.linspace(4, -4, V)
        elif kind == "clustered":
            v = rng.normal(0, 1, V)
            s = rng.integers(0, max(1, V - 30))
            v[s:s + 30] += 9.0
        elif kind == "one_lane":
            v = rng.normal(0, 1, V)
            v[3::1024] += 9.0
            v[7::2048] += 2.0
        elif kind == "masked":
            v = np.full(V, -np.inf)
            v[rng.integers(0, V, 5)] = rng.normal(0, 1, 5)
            if t % 4 == 3:
                v[:] = -np.inf
        elif kind == "zeros":
            v = np.where(rng.random(V) < 0.5, 0.0, -0.0)
        else:
            v = np.full(V, -3.0e38)
            v[rng.integers(0, V, 3)] = 1.0
        rows.append(v)
    for dtype in ("f32", "bf16"):
        x = torch.from_numpy(np.array(rows)).to(TDT[dtype]).cuda()
        run(x, host(x), 33)
        run(x, host(x), min(V, 700))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2, 130])
def test_long_lists_of_the_longest_lined_rows(T, dtype):
    """The most line maxima and the most candidates at once (66 KB of LDS), in parts and in one block."""
    need_gpu()
    V = 262144 if dtype == "f32" else 524288
    x = torch.randn((T, V), device="cuda").to(TDT[dtype])
    idx, logp, lse = sg.sg_topk_rows(x, 1000)
    for t in (0, T - 1):
        ri, rp, rl = ref.topk_rows(host(x[t:t + 1]), 1000, 1.0)
        assert np.array_equal(idx[t:t + 1].cpu().numpy(), ri)
        check(host(logp)[t:t + 1], rp, ref.sum_error(V) + 2.0 ** -24 * np.abs(rp), "logp")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_rows(dtype):
    need_gpu()
    for V, ld, shift in ((1001, 1009, 1), (70001, 70004, 3)):
        x, xs = make_logits(V, 5, V, dtype, ld, shift)
        run(x, xs, 40)


def test_nan_and_infinity_stay_in_their_rows():
    need_gpu()
    x, xs = make_logits(1, 5, 3000, "f32")
    x[1, 77] = float("nan")
    x[3, 88] = float("inf")
    idx, logp, lse = sg.sg_topk_rows(x, 20)
    idx = idx.cpu().numpy()
    assert 77 in idx[1] and 88 in idx[3]
    assert list(np.flatnonzero(np.isnan(host(lse)))) == [1, 3]
    ri, rp, _ = ref.topk_rows(xs, 20, 1.0)
    for t in (0, 2, 4):
        assert np.array_equal(idx[t], ri[t])
        check(host(logp)[t], rp[t], ref.sum_error(3000) + 2.0 ** -24 * np.abs(rp[t]), "logp")


def test_rows_feed_distillation():
    """A student equal to its teacher: the lists of sg_topk_rows give a loss of almost nothing."""
    need_gpu()
    x, xs = make_logits(2, 9, 32000, "bf16")
    idx, logp, _ = sg.sg_topk_rows(x, 64, temperature=2.0)
    loss, grad = sg.sg_distill_loss(x, idx, logp, temperature=2.0)
    # KL of two distributions whose log-masses differ by e is at most of order e^2, computed from terms of order one
    assert host(loss).max() <= 10 * ref.sum_error(32000)
    assert np.abs(host(grad)).max() <= 10 * ref.sum_error(32000)


def test_offsets_beyond_32_bits():
    need_gpu()
    T, V = 33000, 131080
    x = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    tail, xs = make_logits(3, 2, V, "bf16")
    x[-2:] = tail
    idx, logp, lse = sg.sg_topk_rows(x, 16)
    ri, rp, rl = ref.topk_rows(xs, 16, 1.0)
    assert np.array_equal(idx[-2:].cpu().numpy(), ri)
    check(host(lse)[-2:], rl, ref.sum_error(V) + 2.0 ** -24 * np.abs(rl), "lse")
    assert np.array_equal(idx[0].cpu().numpy(), np.arange(16))
