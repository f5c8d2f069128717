"""Definitions in 64 bits of the operators around a step (head's cross entropy,
router's balance, orthogonalised update), and how far a result may be from
them, from the roundings that each operator states.  Runs on whatever device
its inputs are on."""
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step relative to the value
U32 = 2.0 ** -24


def linear_ce(x, w, label, weight, it, zc):
    """Values and elementwise error bounds of (loss, lse, grad_hidden, grad_head)
    as two dicts.  The bounds add up:
      z      H fp32 additions, and for fp32 operands 2^-21 of each product (two
             22-bit planes a factor, the product of the low ones left out)
      lse    the worst z of the row, 2^-22 for exponentials and their sums, its own rounding
      g      twice z's error (its exponential and lse), 2^-20 for the exponential and its scale,
             2^-11 for the kept 16 bits, half a bf16 step; fp32: 2^-20 and 2^-21.  An exponential below
             2^-63 of its tile's largest has no 16-bit number and counts as 0 (fp32: below 2^-126, the
             smallest normal number): at most that much of the row's factor, since no p is above 1
      dx, dw g's errors and V (T) fp32 additions of the products' magnitudes, the output's rounding"""
    dt, H = x.dtype, x.shape[1]
    bf = dt == torch.bfloat16
    V = w.shape[0]
    live = (label >= 0) & (label < V)
    if weight is None:
        weight = torch.ones(x.shape[0], device=x.device)
    live = live & (weight != 0)
    X = torch.where(live[:, None], x.double(), 0.0)
    W = w.double()
    wt = torch.where(live, weight.double(), 0.0)
    y = torch.where(live, label, 0).long()
    z = it * X @ W.t()
    size = it * X.abs() @ W.abs().t()
    ez = size * (H * U32 + (0.0 if bf else 2.0 ** -21)) + z.abs() * 2.0 ** -22
    lse = torch.logsumexp(z, 1)
    elv = ez.amax(1) + 2.0 ** -22 * (1.0 + (z.amax(1)[:, None] - z).amax(1) * 0.25)
    zy = z.gather(1, y[:, None])[:, 0]
    loss = wt * (lse - zy + zc * lse ** 2)
    eloss = wt.abs() * (elv * (1 + 2 * zc * lse.abs()) + ez.gather(1, y[:, None])[:, 0]) + U32 * loss.abs()
    q = torch.exp(z - lse[:, None])
    one = torch.zeros_like(q).scatter_(1, y[:, None], 1.0)
    fac = 1 + 2 * zc * lse
    g = (wt * it)[:, None] * (fac[:, None] * q - one)
    big = (wt.abs() * it)[:, None] * (fac.abs()[:, None] * q + one)
    rel = ez + elv[:, None] + (2.0 ** -20 if not bf else 2.0 ** -20 + 2.0 ** -11)
    eg = (wt.abs() * it)[:, None] * q * (fac.abs()[:, None] * rel + 2 * zc * elv[:, None]) + 2.0 ** -22 * big
    eg = eg + g.abs() * (2.0 ** -8 if bf else 2.0 ** -21)
    eg = eg + (2.0 ** -63 if bf else 2.0 ** -126) * ((wt.abs() * it) * fac.abs())[:, None]
    # the fp16 planes' smallest step, relative to the tensor's largest element
    if not bf:
        eg = eg + 2.0 ** -37 * big.amax()
    dx, dw = g @ W, g.t() @ X
    ab = 0.0 if bf else 2.0 ** -20
    edx = eg @ W.abs() + (V * U32 + ab) * (g.abs() @ W.abs()) + HALF[dt] * dx.abs()
    edw = eg.t() @ X.abs() + (x.shape[0] * U32 + ab) * (g.abs().t() @ X.abs()) + HALF[dt] * dw.abs()
    val = dict(loss=loss, lse=torch.where(live, lse, 0.0), grad_hidden=dx, grad_head=dw)
    err = dict(loss=eloss, lse=torch.where(live, elv + U32 * lse.abs(), 0.0), grad_hidden=edx, grad_head=edw)
    return val, err


def balance(x, idx, live, alpha, zc):
    """Values and bounds of (loss, counts, prob, grad).  p: 2^-21 a row (the
    exponentials of up to 1024 logits within 30 of the largest, their sum, the division); a
    column's sum adds at most 2^-24 for each of the fp32 additions of its block."""
    T, E = x.shape
    k = idx.shape[1]
    if live is None:
        live = torch.ones(T, dtype=torch.bool, device=x.device)
    rows = torch.nonzero(live)[:, 0]
    z = x[rows].double()
    n = max(1, rows.numel())
    flat = idx[rows].reshape(-1).long()
    counts = torch.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
    lse = torch.logsumexp(z, 1)
    p = torch.softmax(z, 1)  # not exp(z - lse): a row at the type's lowest value has lse = z in 64 bits too
    f = counts.double() / (k * n)
    prob = p.sum(0) / n
    loss = alpha * E * (f * prob).sum() + zc * (lse ** 2).sum() / n
    h = alpha * E * f / n
    dot = (p * h).sum(1, keepdim=True)
    grad = torch.zeros((T, E), dtype=torch.float64, device=x.device)
    grad[rows] = p * (h - dot + 2 * zc * lse[:, None] / n)
    spread = (z.amax(1) - z.amin(1).clamp_min(-1e30) if E else lse) if rows.numel() else lse
    ep = 2.0 ** -21 * (1 + spread.clamp_max(88.0) / 8)
    eg = torch.zeros_like(grad)
    eg[rows] = p * ((h + dot + 2 * zc * lse.abs()[:, None] / n) * (ep[:, None] + 2.0 ** -21)) + HALF[x.dtype] * grad[rows].abs()
    worst = float(ep.max()) if rows.numel() else 0.0
    rel = worst + 64 * U32 + min(T, 4096) * U32
    val = dict(loss=loss, counts=counts, prob=prob, grad=grad)
    err = dict(loss=rel * alpha * E * (f * prob).sum() + zc * 2.0 ** -21 * ((lse.abs() + 1) * 2 * lse.abs()).sum() / n + U32 * loss.abs(),
               prob=rel * prob, grad=eg)
    return val, err


def orthogonalize(u, steps, coef, eps, bits=None):
    """The definition; with `bits` every stored matrix is rounded to so many
    significant bits: a model of the roundings that the operator states."""
    a, b, c = coef
    r = (lambda t: t) if bits is None else (lambda t: _round(t, bits))
    x = u.double()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-2, -1)
    x = r((x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)).contiguous())
    for _ in range(steps):
        g = r(x @ x.transpose(-2, -1).contiguous())
        x = r(a * x + r(b * g + c * (g @ g)) @ x)
    return x.transpose(-2, -1).contiguous() if tall else x


def _round(t, bits):
    m, e = torch.frexp(t)
    return torch.ldexp(torch.round(m * 2.0 ** bits), e - bits)


def orthogonalize_error(u, steps, coef, eps):
    """Norm of the error allowed for each matrix: three times what the model with
    the operator's bits is off (11, or 21 of 22 and fp32's sums), and the output's rounding."""
    exact = orthogonalize(u, steps, coef, eps)
    model = orthogonalize(u, steps, coef, eps, 11 if u.dtype == torch.bfloat16 else 21)
    norm = exact.square().sum((-2, -1)).sqrt()
    off = (model - exact).square().sum((-2, -1)).sqrt()
    return exact, 3 * off + (HALF[u.dtype] + 2.0 ** -20) * norm


def close(got, want, bound, what):
    """|got - want| <= bound; what is below the smallest normal fp32 number may be 0."""
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= bound + 2.0 ** -126)
    n = int(bad.sum())
    if n:
        at = torch.nonzero(bad.reshape(-1))[0, 0]
        raise AssertionError("%s: %d of %d out of bounds, first at %d: got %r, want %r, bound %r" % (
            what, n, bad.numel(), int(at), float(got.reshape(-1)[at]), float(want.reshape(-1)[at]),
            float(torch.as_tensor(bound, device=got.device).expand(got.shape).reshape(-1)[at])))
