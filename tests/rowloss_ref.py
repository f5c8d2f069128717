"""The vocabulary losses from their definitions in numpy, 64 bits, one row at
a time, and the error bounds their fp32 kernels are held to.

Every function takes raw logits [T, V] as float64 and returns per-row results;
nothing here shares code with the library."""
import numpy as np


def log_softmax(x, inv_temp):
    """log q of one row; -inf where the logit is -inf, also if all are."""
    z = x * inv_temp
    m = z.max()
    if m == -np.inf:
        return np.full_like(z, -np.inf), -np.inf
    log_sum = np.log(np.exp(z - m).sum())
    return (z - m) - log_sum, m + log_sum  # not z - lse: a row may lie at the type's lowest value


def topk_rows(x, k, inv_temp):
    T, V = x.shape
    idx = np.empty((T, k), np.int64)
    logp = np.empty((T, k))
    lse = np.empty(T)
    for t in range(T):
        order = np.argsort(-x[t], kind="stable")  # equal values stay in index order (-0 == +0)
        idx[t] = np.sort(order[:k])
        lq, lse[t] = log_softmax(x[t], inv_temp)
        logp[t] = lq[idx[t]]
    return idx, logp, lse


def distill_row(x, idx, logp, inv_temp, mode):
    """(L, dL/dx, scale) of one row; scale[i] bounds what the terms of dL/dx[i] add up to in magnitude."""
    V = x.size
    lq, _ = log_softmax(x, inv_temp)
    q = np.exp(lq)
    ok = (idx >= 0) & (idx < V)
    idx, logp = idx[ok], logp[ok]
    p = np.exp(logp)
    P = p.sum()
    W, R = P, 0.0
    if mode == "renorm":
        if P == 0.0:
            return 0.0, np.zeros(V), np.zeros(V)
        logp, p, W = logp - np.log(P), p / P, 1.0
    L = sum((pj * (tj - lq[i]) for i, tj, pj in zip(idx, logp, p) if pj > 0), 0.0)
    g, scale = W * q, W * q
    if mode == "tail":
        others = np.ones(V, bool)
        others[idx] = False
        rest = q[others].sum()
        R = max(0.0, 1.0 - P)
        if rest == 0.0:
            R = 0.0
        if R > 0.0:
            L += R * (np.log(R) - np.log(rest))
        g = (P + R) * q
        scale = g.copy()
        if R > 0.0:
            g[others] -= R / rest * q[others]
            scale[others] += R / rest * q[others]
    np.subtract.at(g, idx, p)
    np.add.at(scale, idx, p)
    return L, inv_temp * g, inv_temp * scale


def policy_row(x, a, old, ref, adv, inv_temp, lo, hi, kl):
    """(L, logp, dL/dx) of one row."""
    lq, _ = log_softmax(x, inv_temp)
    lp = lq[a]
    r = 1.0 if old is None else np.exp(lp - old)
    L = -min(r * adv, np.clip(r, 1 - lo, 1 + hi) * adv)
    s = 0.0 if (adv > 0 and r > 1 + hi) or (adv < 0 and r < 1 - lo) else -r * adv
    if ref is not None:
        d = ref - lp
        L += kl * (np.exp(d) - d - 1)
        s += kl * (1 - np.exp(d))
    e = np.zeros(x.size)
    e[a] = 1.0
    return L, lp, s * inv_temp * (e - np.exp(lq))


def preference(x, label, off, ref, weight, kind, beta, eps, average):
    """(loss [B], S [2B], dloss/dx [T, V])."""
    T, V = x.shape
    B = (len(off) - 1) // 2
    lq = [log_softmax(x[t], 1.0)[0] for t in range(T)]
    counts = [(0 <= label[t] < V) for t in range(T)]
    S, n = np.zeros(2 * B), np.ones(2 * B)
    for s in range(2 * B):
        rows = [t for t in range(off[s], off[s + 1]) if counts[t]]
        S[s] = sum(lq[t][label[t]] for t in rows)
        if average:
            n[s] = max(1, len(rows))
        S[s] /= n[s]
    grad = np.zeros((T, V))
    loss = np.zeros(B)
    for b in range(B):
        d = (S[b] - ref[b]) - (S[B + b] - ref[B + b])
        if kind == "ipo":
            L, g = (d - 0.5 / beta) ** 2, 2 * (d - 0.5 / beta)
        elif kind == "hinge":
            L, g = max(0.0, 1 - beta * d), (-beta if beta * d < 1 else 0.0)
        else:
            h = beta * d
            L = (1 - eps) * np.logaddexp(0, -h) + eps * np.logaddexp(0, h)
            g = beta * (eps / (1 + np.exp(-h)) - (1 - eps) / (1 + np.exp(h)))
        loss[b] = weight[b] * L
        for s, sign in ((b, 1.0), (B + b, -1.0)):
            for t in range(off[s], off[s + 1]):
                if counts[t]:
                    e = np.zeros(V)
                    e[label[t]] = 1.0
                    grad[t] = sign * weight[b] * g / n[s] * (e - np.exp(lq[t]))
    return loss, S, grad


HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def sum_error(V):
    """Bound of the relative error of a row's sum of exponentials.  Each term
    has the rounding of the difference, of its product with log2(e)/temperature
    (and of that constant) and of the exponential: an exponent of size a is off
    by at most 3 * 2^-24 a, and a term that matters has a <= 32 (e^-22 of the
    maximum times any V here is below the bound), the instruction itself by one
    unit, 2^-23.  A lane adds at most V / 256 + 16 terms one after the other
    (half a unit each), the join takes at most 24 more steps, each with two
    exponentials of its own."""
    return 3 * 32 * 2.0 ** -24 + 2.0 ** -23 + (V / 256 + 16) * 2.0 ** -24 + 24 * 4 * 2.0 ** -23


def grad_error(V, depth):
    """Bound of the relative error of one term of the gradient at `depth`
    (scaled distance of the logit below the row's maximum) before its rounding:
    the sum's, and the exponential's at that depth."""
    return sum_error(V) + 3 * 1.4427 * depth * 2.0 ** -24 + 2.0 ** -22
