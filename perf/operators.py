"""The losses over a vocabulary that a data-parallel step starts from, and the
teacher's side of distillation, as measured cases.

Four operators of ``sparse_gradient_synchronization_amd``:

  topk_rows   the k largest logits of every row as COO rows (ascending
              indices) with their log-probabilities: what a teacher sends
  distill     the divergence of a student's logits from such rows, with the
              gradient with respect to the logits
  policy      a clipped policy-ratio loss with a KL term to a reference, per
              token, with its gradient
  preference  a paired log-ratio loss over packed sequences, with its gradient

Every case is one call of one of them.  ``own`` says whether ``run`` makes
that call or computes the plain form with elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_ESIZE = {"f32": 4, "bf16": 2}


def _case(name, op, T, V, dtype, **more):
    c = {"name": name, "op": op, "T": T, "V": V, "dtype": dtype, "pad": 0}
    c.update(more)
    return c


def listed():
    return [
        # a teacher answering for a handful of tokens, as it does while it generates: latency
        _case("topk-few", "topk_rows", 4, 32000, "f32", k=20, temperature=1.0),
        # a batch of an odd vocabulary in fp32; no row but the first starts on 16 bytes
        _case("topk-odd", "topk_rows", 1500, 50001, "f32", k=64, temperature=2.0),
        # the teacher's pass over a whole training batch, long lists
        _case("topk-batch", "topk_rows", 8192, 131072, "bf16", k=128, temperature=1.0),
        # one short sequence, student in bf16
        _case("distill-few", "distill", 24, 32000, "bf16", k=16, temperature=1.0, mode="tail", masked=0.0, grad=True),
        # the evaluation loss of an fp32 student, the vocabulary padded to a wider row
        _case("distill-eval", "distill", 2000, 50021, "f32", k=50, temperature=2.0, mode="renorm", masked=0.25,
              grad=False, pad=43),
        # a training batch: loss and gradient in one call
        _case("distill-train", "distill", 6000, 131072, "bf16", k=64, temperature=1.0, mode="tail", masked=0.1,
              grad=True),
        # the tokens of one short answer
        _case("policy-few", "policy", 7, 65536, "bf16", temperature=1.0, kl=0.05, masked=0.0, grad=True),
        # log-probabilities and loss without gradient (old policy, monitoring), odd vocabulary
        _case("policy-eval", "policy", 4096, 100003, "bf16", temperature=0.8, kl=0.02, masked=0.3, grad=False),
        # a training batch; the prompts' tokens carry no weight
        _case("policy-train", "policy", 8192, 131072, "bf16", temperature=1.0, kl=0.05, masked=0.3, grad=True),
        # two pairs of short answers, fp32
        _case("preference-few", "preference", 90, 32000, "f32", pairs=2, kind="sigmoid", average=False, masked=0.2,
              grad=True),
        # the reference model's pass: summed log-probabilities only
        _case("preference-eval", "preference", 5000, 65536, "bf16", pairs=24, kind="sigmoid", average=False,
              masked=0.4, grad=False),
        # a training batch of pairs, length-normalised
        _case("preference-train", "preference", 6000, 131072, "bf16", pairs=16, kind="ipo", average=True, masked=0.3,
              grad=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["topk_rows", "distill", "policy", "preference"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    V = _log_int(rng, 500, 260000)
    if rng.random() < 0.5:  # half of the vocabularies are multiples of 64, the others whatever comes
        V = max(512, V // 64 * 64)
    most = 6000 * 131072 * 2 // _ESIZE[dtype]
    T = _log_int(rng, 1, max(1, min(16384, most // V)))
    c = {"op": op, "T": T, "V": V, "dtype": dtype, "pad": rng.choice([0, 0, rng.randrange(1, 128)])}
    if op == "topk_rows":
        c.update(k=min(V, _log_int(rng, 1, 256)), temperature=rng.choice([1.0, 1.0, 2.0, 0.5]))
        return c
    c.update(masked=rng.choice([0.0, round(rng.uniform(0, 0.6), 3)]), grad=rng.random() < 0.7)
    if op == "distill":
        c.update(k=min(V, _log_int(rng, 1, 256)), temperature=rng.choice([1.0, 2.0, 4.0]),
                 mode=rng.choice(["tail", "renorm", "plain"]))
    elif op == "policy":
        c.update(temperature=rng.choice([1.0, 0.7, 1.3]), kl=rng.choice([0.0, 0.02, 0.1]))
    else:
        c.update(pairs=_log_int(rng, 1, max(1, min(64, T))), kind=rng.choice(["sigmoid", "hinge", "ipo"]),
                 average=rng.random() < 0.5)
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
_BOOSTED = 8  # likely tokens per row


def _logits(case, g):
    """[T, V] logits in a buffer of V + pad columns: rows of differing
    sharpness with a few likely tokens each.  Returns (logits, likely [T, 8])."""
    T, V = case["T"], case["V"]
    x = torch.randn((T, V + case["pad"]), device="cuda", generator=g)
    x *= 1.0 + 1.5 * torch.rand((T, 1), device="cuda", generator=g)
    likely = torch.randint(0, V, (T, _BOOSTED), device="cuda", generator=g)
    top = 4.0 + 8.0 * torch.rand((T, _BOOSTED), device="cuda", generator=g)
    x.scatter_(1, likely, top)
    return x.to(_DTYPES[case["dtype"]])[:, :V], likely


def _weights(case, g):
    """Per-token weights: zero for the masked share, 1 / (rows that count) otherwise."""
    T = case["T"]
    off = int(T * case["masked"])
    w = torch.full((T,), 1.0 / max(1, T - off), device="cuda")
    w[torch.randperm(T, device="cuda", generator=g)[:off]] = 0.0
    return w


def _tokens(likely, V, g):
    """One token per row, mostly a likely one."""
    T = likely.shape[0]
    pick = likely.gather(1, torch.randint(0, _BOOSTED, (T, 1), device="cuda", generator=g))[:, 0]
    other = torch.randint(0, V, (T,), device="cuda", generator=g)
    return torch.where(torch.rand(T, device="cuda", generator=g) < 0.85, pick, other)


def _token_logp(logits, token, scale):
    z = logits.float() * scale
    return z.gather(1, token[:, None])[:, 0] - torch.logsumexp(z, 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    T, V, op = case["T"], case["V"], case["op"]
    logits, likely = _logits(case, g)
    s = {"case": dict(case), "logits": logits}
    if op == "topk_rows":
        return s
    if op == "distill":
        k, temp = case["k"], case["temperature"]
        s["weight"] = _weights(case, g)
        teacher = torch.randn((T, V), device="cuda", generator=g).add_(logits, alpha=0.8)
        val, idx = torch.topk(teacher, k, dim=1)
        logp = val / temp - torch.logsumexp(teacher / temp, 1, keepdim=True)
        # a fifth of the lists is shorter: their last places are padding
        short = torch.rand((T, 1), device="cuda", generator=g) < 0.2
        kept = torch.randint(0, k + 1, (T, 1), device="cuda", generator=g)
        idx = torch.where(short & (torch.arange(k, device="cuda") >= kept), -1, idx)
        s["idx"], s["logp"] = idx.to(torch.int32).contiguous(), logp.contiguous()
    elif op == "policy":
        s["weight"] = _weights(case, g)
        token = _tokens(likely, V, g)
        logp = _token_logp(logits, token, 1.0 / case["temperature"])
        s["action"] = token.to(torch.int32)
        s["old"] = logp + 0.15 * torch.randn(T, device="cuda", generator=g)
        s["ref"] = logp + 0.3 * torch.randn(T, device="cuda", generator=g) if case["kl"] > 0 else None
        s["adv"] = torch.randn(T, device="cuda", generator=g)
    else:
        B = case["pairs"]
        token = _tokens(likely, V, g)
        live = torch.ones(T, dtype=torch.bool, device="cuda")
        live[torch.randperm(T, device="cuda", generator=g)[:int(T * case["masked"])]] = False
        cuts = torch.randint(0, T + 1, (2 * B - 1,), device="cuda", generator=g).sort().values
        s["off"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)])
        logp = _token_logp(logits, token, 1.0).double() * live
        total = torch.cat([logp.new_zeros(1), logp.cumsum(0)])[s["off"]].diff()
        lens = (s["off"].diff().double()).clamp_min(1.0)
        # the reference agrees up to a few nats, whatever the length
        s["ref"] = ((total / lens if case["average"] else total)
                    + torch.randn(2 * B, device="cuda", generator=g).double() * (0.2 if case["average"] else 3.0)).float()
        s["label"] = torch.where(live, token, -1).to(torch.int32)
        s["weight"] = torch.full((B,), 1.0 / B, device="cuda")
    return s


_BETA = 0.1
_SMOOTHING = 0.05
_CLIP = (0.2, 0.28)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _softmax_parts(logits, scale):
    """z = scale * logits in fp32, row maximum, exp(z - max), its sum in fp64, lse in fp64."""
    z = logits.float() * scale
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    tot = e.sum(1, keepdim=True, dtype=torch.float64)
    return z, m, e, tot, m.double() + torch.log(tot)


def _plain_topk(s):
    c, x = s["case"], s["logits"]
    V = c["V"]
    z, _, _, _, lse = _softmax_parts(x, 1.0 / c["temperature"])
    bits = (x.float() + 0.0).view(torch.int32)  # + 0.0 makes -0 the same as +0
    order = (bits ^ ((bits >> 31) & 0x7fffffff)).long()
    key = (order << 32) | (V - 1 - torch.arange(V, device=x.device))  # ties go to the lowest index
    idx = (V - 1 - (torch.topk(key, c["k"], dim=1).values & 0xffffffff)).sort(1).values
    return idx.to(torch.int32), (z.gather(1, idx).double() - lse).float(), lse[:, 0].float()


def _plain_distill(s):
    c, x, w = s["case"], s["logits"], s["weight"].double()[:, None]
    V, scale = c["V"], 1.0 / c["temperature"]
    z, m, e, tot, lse = _softmax_parts(x, scale)
    valid = (s["idx"] >= 0) & (s["idx"] < V)
    at = torch.where(valid, s["idx"], 0).long()
    t = s["logp"].double()
    p = torch.where(valid, torch.exp(t), 0.0)
    mass = p.sum(1, keepdim=True)
    tail = torch.zeros_like(mass)
    if c["mode"] == "renorm":
        t = t - torch.log(mass)
        p = torch.where(mass > 0, p / mass, 0.0)
        mass = torch.where(mass > 0, 1.0, 0.0)
    elif c["mode"] == "tail":
        tail = (1.0 - mass).clamp_min(0.0)
    loss = torch.where(p > 0, p * (t - z.gather(1, at).double() + lse), 0.0).sum(1, keepdim=True)
    within = (mass + tail) / tot  # the factor of e in the gradient, for listed tokens and for the others
    rest = within
    if c["mode"] == "tail":
        listed_ = torch.zeros((x.shape[0], V + 1), dtype=torch.bool, device=x.device)
        listed_.scatter_(1, torch.where(valid, s["idx"], V).long(), True)
        other = e.masked_fill(listed_[:, :V], 0.0).sum(1, keepdim=True, dtype=torch.float64)
        has = (other > 0) & (tail > 0)
        tail = torch.where(has, tail, 0.0)
        loss = loss + torch.where(has, tail * (torch.log(tail) + torch.log(tot / other)), 0.0)
        within = (mass + tail) / tot
        rest = within - torch.where(has, tail / other, 0.0)
    live = w != 0
    loss = torch.where(live, w * loss, 0.0)[:, 0].float()
    if not c["grad"]:
        return loss
    gw = torch.where(live, w * scale, 0.0)
    if c["mode"] == "tail":
        grad = e * torch.where(listed_[:, :V], (gw * within).float(), (gw * rest).float())
    else:
        grad = e * (gw * within).float()
    grad.scatter_add_(1, at, torch.where(valid, -gw * p, 0.0).float())
    return loss, grad.to(x.dtype)


def _plain_policy(s):
    c, x, w = s["case"], s["logits"], s["weight"].double()
    scale = 1.0 / c["temperature"]
    z, m, e, tot, lse = _softmax_parts(x, scale)
    a = s["action"].long()[:, None]
    logp = z.gather(1, a)[:, 0].double() - lse[:, 0]
    adv = s["adv"].double()
    r = torch.exp(logp - s["old"].double())
    loss = -torch.minimum(r * adv, r.clamp(1.0 - _CLIP[0], 1.0 + _CLIP[1]) * adv)
    clipped = ((adv > 0) & (r > 1.0 + _CLIP[1])) | ((adv < 0) & (r < 1.0 - _CLIP[0]))
    slope = torch.where(clipped, 0.0, -adv * r)
    if s["ref"] is not None:
        d = s["ref"].double() - logp
        loss = loss + c["kl"] * (torch.expm1(d) - d)
        slope = slope - c["kl"] * torch.expm1(d)
    live = w != 0
    loss = torch.where(live, w * loss, 0.0).float()
    logp = torch.where(live, logp, 0.0)
    if not c["grad"]:
        return loss, logp.float()
    slope = torch.where(live, w * slope * scale, 0.0)[:, None]
    grad = e * (-slope / tot).float()
    grad.scatter_(1, a, (slope * -torch.expm1(logp[:, None])).float())
    return loss, logp.float(), grad.to(x.dtype)


def _plain_preference(s):
    c, x, w = s["case"], s["logits"], s["weight"].double()
    B, T = c["pairs"], c["T"]
    z, m, e, tot, lse = _softmax_parts(x, 1.0)
    live = (s["label"] >= 0) & (s["label"] < c["V"])
    y = torch.where(live, s["label"], 0).long()[:, None]
    logp = torch.where(live, z.gather(1, y)[:, 0].double() - lse[:, 0], 0.0)
    seq = torch.searchsorted(s["off"], torch.arange(T, device=x.device), right=True) - 1
    total = torch.zeros(2 * B, dtype=torch.float64, device=x.device).index_add_(0, seq, logp)
    per = torch.ones_like(total)
    if c["average"]:
        per = torch.zeros_like(total).index_add_(0, seq, live.double()).clamp_min(1.0)
        total = total / per
    d = total - s["ref"].double()
    d = d[:B] - d[B:]
    if c["kind"] == "ipo":
        gap = d - 0.5 / _BETA
        loss, slope = gap * gap, 2.0 * gap
    elif c["kind"] == "hinge":
        loss, slope = (1.0 - _BETA * d).clamp_min(0.0), torch.where(_BETA * d < 1.0, -_BETA, 0.0)
    else:
        h = _BETA * d
        up, down = torch.log1p(torch.exp(-h.abs())) + (-h).clamp_min(0.0), torch.log1p(torch.exp(-h.abs())) + h.clamp_min(0.0)
        loss = (1.0 - _SMOOTHING) * up + _SMOOTHING * down
        slope = _BETA * (_SMOOTHING * torch.exp(-up) - (1.0 - _SMOOTHING) * torch.exp(-down))
    loss = (w * loss).float()
    if not c["grad"]:
        return loss, total.float()
    slope = torch.cat([w * slope, -w * slope]) / per
    slope = torch.where(live, slope[seq], 0.0)[:, None]
    grad = e * (-slope / tot).float()
    grad.scatter_(1, y, torch.where(live[:, None], slope * -torch.expm1(logp[:, None]), 0.0).float())
    return loss, total.float(), grad.to(x.dtype)


_PLAIN = {"topk_rows": _plain_topk, "distill": _plain_distill, "policy": _plain_policy,
          "preference": _plain_preference}


def _call(s):
    import sparse_gradient_synchronization_amd as sg
    c, x = s["case"], s["logits"]
    if c["op"] == "topk_rows":
        return sg.sg_topk_rows(x, c["k"], temperature=c["temperature"])
    if c["op"] == "distill":
        mode = {"tail": sg.SG_DISTILL_TAIL, "renorm": sg.SG_DISTILL_RENORM, "plain": sg.SG_DISTILL_PLAIN}[c["mode"]]
        loss, grad = sg.sg_distill_loss(x, s["idx"], s["logp"], temperature=c["temperature"], mode=mode,
                                        weight=s["weight"], want_grad=c["grad"])
        return (loss, grad) if c["grad"] else loss
    if c["op"] == "policy":
        loss, logp, grad = sg.sg_policy_loss(x, s["action"], s["old"], s["adv"], ref_logp=s["ref"], weight=s["weight"],
                                             clip_low=_CLIP[0], clip_high=_CLIP[1], kl_coef=c["kl"],
                                             temperature=c["temperature"], want_grad=c["grad"])
    else:
        kind = {"sigmoid": sg.SG_PREF_SIGMOID, "hinge": sg.SG_PREF_HINGE, "ipo": sg.SG_PREF_IPO}[c["kind"]]
        loss, logp, grad = sg.sg_preference_loss(x, s["label"], s["off"], ref_logp=s["ref"], weight=s["weight"],
                                                 kind=kind, beta=_BETA, smoothing=_SMOOTHING, average=c["average"],
                                                 want_grad=c["grad"])
    return (loss, logp, grad) if c["grad"] else (loss, logp)


def run(state):
    return _call(state) if own else _PLAIN[state["case"]["op"]](state)


def work(case):
    """The logits of the rows that count read once, the whole gradient written
    once, and the lists; three operations an element for the sum of the
    exponentials and two for the gradient."""
    T, V, e = case["T"], case["V"], _ESIZE[case["dtype"]]
    live = T - int(T * case.get("masked", 0.0))
    nbytes, flops = live * V * e, 3 * live * V
    if case["op"] == "topk_rows":
        nbytes, flops = nbytes + T * (8 * case["k"] + 4), flops + T * V
    elif case["op"] == "distill":
        nbytes += live * 8 * case["k"] + 8 * T
    else:
        nbytes += 28 * T
    if case.get("grad"):
        nbytes, flops = nbytes + T * V * e, flops + 2 * live * V
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
_ROWS = 1 << 26  # elements of a slab of rows


def _slabs(case):
    step = max(1, _ROWS // case["V"])
    return [slice(a, min(a + step, case["T"])) for a in range(0, case["T"], step)]


def _log_softmax64(x, temperature):
    z = x.double() / temperature
    return z - torch.logsumexp(z, 1, keepdim=True)


def exact(case, seed):
    s = prepare(case, seed)
    x, op = s["logits"], case["op"]
    T, V = case["T"], case["V"]
    slabs = _slabs(case)
    if op == "topk_rows":
        logp, lse = [], []
        for r in slabs:
            z = x[r].double() / case["temperature"]
            first = torch.sort(x[r].double(), dim=1, descending=True, stable=True).indices[:, :case["k"]].sort(1).values
            lse.append(torch.logsumexp(z, 1))
            logp.append(z.gather(1, first) - lse[-1][:, None])
        return None, torch.cat(logp), torch.cat(lse)

    grad = torch.zeros((T, V), dtype=torch.float64, device=x.device) if case["grad"] else None
    if op == "distill":
        loss = torch.zeros(T, dtype=torch.float64, device=x.device)
        for r in slabs:
            w = s["weight"][r].double()
            lq = _log_softmax64(x[r], case["temperature"])
            q = lq.exp()
            # the teacher's masses laid out over the vocabulary, one more column taking the padding
            valid = (s["idx"][r] >= 0) & (s["idx"][r] < V)
            dense = torch.zeros((q.shape[0], V + 1), dtype=torch.float64, device=x.device)
            dense.scatter_(1, torch.where(valid, s["idx"][r].long(), V), s["logp"][r].double().exp())
            named = torch.zeros((q.shape[0], V + 1), dtype=torch.bool, device=x.device)
            named.scatter_(1, torch.where(valid, s["idx"][r].long(), V), True)
            p, named = dense[:, :V], named[:, :V]
            total = p.sum(1, keepdim=True)
            if case["mode"] == "renorm":
                p = torch.where(total > 0, p / total, 0.0)
                total = (total > 0).double()
            loss[r] = w * (torch.xlogy(p, p) - p * lq).sum(1)
            dz = q * total - p
            if case["mode"] == "tail":
                left = (1.0 - total).clamp_min(0.0)
                q_left = torch.where(named, 0.0, q).sum(1, keepdim=True)
                left = torch.where(q_left > 0, left, 0.0)
                loss[r] += w * (torch.xlogy(left, left) - torch.xlogy(left, q_left))[:, 0]
                dz = dz + q * left - torch.where(named, 0.0, q * torch.where(left > 0, left / q_left, 0.0))
            if grad is not None:
                grad[r] = w[:, None] * dz / case["temperature"]
        return loss if grad is None else (loss, grad)

    if op == "policy":
        token, temp = s["action"].long(), case["temperature"]
        logp = torch.cat([_log_softmax64(x[r], temp).gather(1, token[r, None])[:, 0] for r in slabs])
        w, adv = s["weight"].double(), s["adv"].double()
        ratio = (logp - s["old"].double()).exp()
        lo, hi = 1.0 - _CLIP[0], 1.0 + _CLIP[1]
        a, b = ratio * adv, ratio.clamp(lo, hi) * adv
        loss = -torch.minimum(a, b)
        d_logp = torch.where(a <= b, -a, 0.0)  # where b is the smaller one it is constant
        if s["ref"] is not None:
            gap = s["ref"].double() - logp
            loss = loss + case["kl"] * (gap.exp() - gap - 1.0)
            d_logp = d_logp + case["kl"] * (1.0 - gap.exp())
        loss, d_logp = w * loss, w * d_logp / temp
        shown = torch.where(w != 0, logp, 0.0)
        out = (loss, shown)
    else:
        token, temp = s["label"].long(), 1.0
        counts = token >= 0
        logp = torch.cat([_log_softmax64(x[r], 1.0).gather(1, token[r, None].clamp_min(0))[:, 0] for r in slabs])
        off, lp = s["off"].cpu().numpy(), (logp * counts).cpu().numpy()
        n = counts.double().cpu().numpy()
        B = case["pairs"]
        total = np.array([lp[a:b].sum() for a, b in zip(off[:-1], off[1:])])
        size = np.array([max(n[a:b].sum(), 1.0) for a, b in zip(off[:-1], off[1:])])
        if not case["average"]:
            size = np.ones_like(size)
        total = total / size
        ratio = total - s["ref"].double().cpu().numpy()
        delta = ratio[:B] - ratio[B:]
        w = s["weight"].double().cpu().numpy()
        if case["kind"] == "ipo":
            loss, slope = (delta - 1.0 / (2.0 * _BETA)) ** 2, 2.0 * (delta - 1.0 / (2.0 * _BETA))
        elif case["kind"] == "hinge":
            loss, slope = np.maximum(0.0, 1.0 - _BETA * delta), -_BETA * (1.0 - _BETA * delta > 0)
        else:
            h = _BETA * delta
            loss = (1.0 - _SMOOTHING) * np.logaddexp(0.0, -h) + _SMOOTHING * np.logaddexp(0.0, h)
            slope = _BETA * (-(1.0 - _SMOOTHING) * np.exp(-np.logaddexp(0.0, h)) + _SMOOTHING * np.exp(-np.logaddexp(0.0, -h)))
        each = np.repeat(np.concatenate([w * slope, -w * slope]) / size, np.diff(off))
        d_logp = torch.from_numpy(each).to(x.device) * counts
        out = (torch.from_numpy(w * loss), torch.from_numpy(total))
    if grad is None:
        return out
    for r in slabs:
        grad[r] = -d_logp[r, None] * _log_softmax64(x[r], temp).exp()
        grad[r].scatter_add_(1, token[r, None].clamp_min(0), d_logp[r, None])
    return out + (grad,)
