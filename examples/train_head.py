"""Trains a vocabulary head on n simulated data-parallel workers of one GPU:
every worker's loss over the vocabulary gives its dense gradient, and the
sparse synchronization path of the library turns the n gradients into one
update.

  python examples/train_head.py [--steps 12] [--loss distill|policy|preference|cross_entropy]
                                [--update sgd|orthogonal]

  loss      distill     sg_topk_rows on a teacher's logits, sg_distill_loss on
                        the workers'
            policy      sg_policy_loss on sampled tokens whose advantage is the
                        teacher's opinion of them
            preference  sg_preference_loss on pairs of token sequences, the
                        teacher's favourites chosen
            cross_entropy  sg_linear_ce_loss on hidden states and the
                        teacher's favourites: the head's gradient without
                        any logits
  gradient  d loss / d head = d loss / d logits ^T  hidden states
  sync      sg_topk_to_coo -> sg_hash_partition -> sg_aggregate ->
            sg_scatter_dense, the largest 5% of every worker's gradient with
            the rest kept for the next step
  update    sgd         the sum of the gradients
            orthogonal  sg_orthogonalize of their momentum, as the Muon
                        optimiser does
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import sparse_gradient_synchronization_amd as sg  # noqa: E402


def synchronize(grads, resid, density, P=4, seed=7):
    """Sum over the workers of the largest `density` of each one's gradient;
    what is not sent stays in resid.  grads, resid [n, M] float32."""
    n, M = grads.shape
    k = max(1, int(M * density))
    total = grads + resid
    idx, val = sg.sg_topk_to_coo(total, k)
    resid.copy_(total)
    resid.scatter_(1, idx.long(), 0.0)
    off = torch.arange(n + 1, device=grads.device) * k
    part_idx, part_val, part_off = sg.sg_hash_partition(idx.reshape(-1), val.reshape(-1), off, P, seed)
    agg_idx, agg_val, agg_off = sg.sg_aggregate(part_idx, part_val, part_off, M)
    return sg.sg_scatter_dense(agg_idx, agg_val, agg_off, M)


def distill_step(logits, teacher, batch, g):
    idx, logp, _ = sg.sg_topk_rows(teacher, 32, temperature=2.0)
    weight = torch.full((logits.shape[0],), 1.0 / logits.shape[0], device=logits.device)
    loss, grad = sg.sg_distill_loss(logits, idx, logp, temperature=2.0, weight=weight, grad=logits)
    return loss.sum(), grad


def policy_step(logits, teacher, batch, g):
    T = logits.shape[0]
    action = torch.multinomial(torch.softmax(logits.float(), 1), 1, generator=g)
    opinion = torch.log_softmax(teacher.float(), 1).gather(1, action)[:, 0]
    adv = (opinion - opinion.mean()) / (opinion.std() + 1e-6)
    action = action[:, 0].int()
    _, old, _ = sg.sg_policy_loss(logits, action, want_grad=False)
    weight = torch.full((T,), 1.0 / T, device=logits.device)
    _, _, grad = sg.sg_policy_loss(logits, action, old, adv, ref_logp=old, weight=weight, kl_coef=0.01, grad=logits)
    return -(opinion.mean()), grad


def preference_step(logits, teacher, batch, g):
    T = logits.shape[0]
    pairs = 8
    off = torch.arange(2 * pairs + 1, device=logits.device) * (T // (2 * pairs))
    # the first half of the rows are chosen sequences, the second half rejected ones
    best, worst = teacher.float().argmax(1), teacher.float().argmin(1)
    label = torch.where(torch.arange(T, device=logits.device) < T // 2, best, worst).int()
    weight = torch.full((pairs,), 1.0 / pairs, device=logits.device)
    loss, _, grad = sg.sg_preference_loss(logits, label, off, weight=weight, beta=0.1, average=True, grad=logits)
    return loss.sum(), grad


def cross_entropy_step(hidden, head, target):
    """(loss, gradient of the head) from hidden states, without logits."""
    label = (hidden @ target.t()).argmax(1).int()
    weight = torch.full((hidden.shape[0],), 1.0 / hidden.shape[0], device=hidden.device)
    loss, _, _, grad = sg.sg_linear_ce_loss(hidden, head, label, weight=weight, want_grad=False,
                                            grad_head=torch.empty_like(head))
    return loss.sum(), grad


STEPS = {"distill": distill_step, "policy": policy_step, "preference": preference_step}


def train(loss="distill", steps=12, workers=4, rows=256, vocab=2000, width=64, density=0.05, rate=None, seed=1,
          update_kind="sgd"):
    """Returns the mean loss of every step (policy: minus the teacher's mean
    log-probability of the sampled tokens)."""
    if rate is None:
        rate = {"distill": 160.0, "policy": 60.0, "preference": 400.0, "cross_entropy": 60.0}[loss]
        if update_kind == "orthogonal":
            rate = 2.0  # singular values near 1, whatever the gradient's size
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    target = torch.randn(vocab, width, device=dev, generator=g) * 0.4
    head = torch.randn(vocab, width, device=dev, generator=g) * 0.05
    resid = torch.zeros(workers, vocab * width, device=dev)
    momentum = torch.zeros_like(head)
    curve = []
    for step in range(steps):
        grads, losses = torch.empty_like(resid), []
        for w in range(workers):
            hidden = torch.randn(rows, width, device=dev, generator=g)
            if loss == "cross_entropy":
                value, grad = cross_entropy_step(hidden, head, target)
                grads[w] = grad.reshape(-1)
                losses.append(value)
                continue
            logits = (hidden @ head.t()).bfloat16()
            teacher = (hidden @ target.t()).bfloat16()
            value, grad = STEPS[loss](logits, teacher, hidden, g)
            grads[w] = (grad.float().t().contiguous() @ hidden).reshape(-1)
            losses.append(value)
        update = synchronize(grads, resid, density).view(vocab, width)
        if update_kind == "orthogonal":
            momentum.mul_(0.9).add_(update)
            head -= rate * sg.sg_orthogonalize(momentum)
        else:
            head -= rate / workers * update
        curve.append(torch.stack(losses).mean())
    return [float(v) for v in torch.stack(curve).cpu()]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--loss", choices=sorted(STEPS) + ["cross_entropy"], default=None,
                    help="default: each in turn")
    ap.add_argument("--update", choices=["sgd", "orthogonal"], default="sgd")
    ap.add_argument("--steps", type=int, default=12)
    a = ap.parse_args()
    for loss in [a.loss] if a.loss else sorted(STEPS) + ["cross_entropy"]:
        curve = train(loss, a.steps, update_kind=a.update)
        print("%-10s %s" % (loss, " ".join("%.4f" % v for v in curve)))
        if sg.sg_device_error():
            raise SystemExit("a kernel noticed a violated precondition")


if __name__ == "__main__":
    main()
