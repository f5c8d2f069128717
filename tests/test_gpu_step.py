"""The operators around a step together, as a data-parallel step uses them:
routers' choices and balance, the head's cross entropy, the gradients through
the sparse synchronization, the update orthogonalised; each stage against its
definition in 64 bits on what the stage before gave it."""
import os
import sys

import pytest
import torch

import sparse_gradient_synchronization_amd as sg
import step_ref as ref
from gpu_util import need_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))

pytestmark = pytest.mark.gpu
COEF = (3.4445, -4.7750, 2.0315)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_step(dtype):
    need_gpu()
    import train_head
    g = torch.Generator(device="cuda").manual_seed(3)
    workers, T, V, H, E = 3, 150, 700, 96, 24
    head = (torch.randn((V, H), device="cuda", generator=g) * 0.2).to(dtype)
    router = torch.randn((E, H), device="cuda", generator=g) * 0.2
    resid_w = torch.zeros((workers, V * H), device="cuda")
    resid_r = torch.zeros((workers, E * H), device="cuda")
    for step in range(3):
        gw, gr = torch.empty_like(resid_w), torch.empty_like(resid_r)
        for w in range(workers):
            x = torch.randn((T, H), device="cuda", generator=g).to(dtype)
            label = torch.randint(-20, V, (T,), device="cuda", generator=g, dtype=torch.int32)
            live = label >= 0
            weight = live.float() / live.sum()
            logits = (x.float() @ router.t()).to(dtype)
            idx, _, _ = sg.sg_topk_rows(logits, 2)
            bal = sg.sg_balance_loss(logits, idx, live=live, balance_coef=0.01, z_coef=1e-3)
            ce = sg.sg_linear_ce_loss(x, head, label, weight=weight, z_coef=1e-4)
            val, err = ref.balance(logits, idx, live, 0.01, 1e-3)
            assert torch.equal(bal[1].long(), val["counts"])
            ref.close(bal[0], val["loss"], err["loss"], "balance")
            ref.close(bal[3], val["grad"], err["grad"], "its gradient")
            val, err = ref.linear_ce(x, head, label, weight, 1.0, 1e-4)
            for name, got in zip(("loss", "lse", "grad_hidden", "grad_head"), ce):
                ref.close(got, val[name], err[name], name)
            gw[w] = ce[3].float().reshape(-1)
            gr[w] = (bal[3].float().t().contiguous() @ x.float()).reshape(-1)
        for grads, resid, weight_, shape in ((gw, resid_w, head, (V, H)), (gr, resid_r, router, (E, H))):
            total = (grads + resid).double().sum(0)
            update = train_head.synchronize(grads, resid, 0.2)
            # what was sent and what was kept is what there was
            assert torch.allclose(update.double() + resid.double().sum(0), total, rtol=1e-5, atol=1e-9)
            u = update.view(shape).to(weight_.dtype)
            want, bound = ref.orthogonalize_error(u, 5, COEF, 1e-7)
            out = sg.sg_orthogonalize(u)
            assert float((out.double() - want).norm()) <= float(bound)
            weight_ -= (0.05 * out.float()).to(weight_.dtype)
            assert bool(torch.isfinite(weight_).all())
    assert sg.sg_device_error() == 0


@pytest.mark.parametrize("kind", ["sgd", "orthogonal"])
@pytest.mark.parametrize("loss", ["cross_entropy", "distill"])
def test_the_example_runs(loss, kind):
    need_gpu()
    import train_head
    curve = train_head.train(loss, steps=3, update_kind=kind)
    assert len(curve) == 3 and all(v == v and abs(v) < 1e3 for v in curve)
    assert sg.sg_device_error() == 0


def test_the_example_gradient():
    """The example's head gradient without logits against the formula's."""
    need_gpu()
    import train_head
    g = torch.Generator(device="cuda").manual_seed(5)
    hidden, head, target = (torch.randn((n, 64), device="cuda", generator=g) * 0.3 for n in (90, 400, 400))
    _, grad = train_head.cross_entropy_step(hidden, head, target)
    label = (hidden @ target.t()).argmax(1).int()
    val, err = ref.linear_ce(hidden, head, label, torch.full((90,), 1.0 / 90, device="cuda"), 1.0, 0.0)
    ref.close(grad, val["grad_head"], err["grad_head"], "grad_head")
