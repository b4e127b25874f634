"""The distillation step of examples/qad_step.py: its gradients against automatic differentiation
in 64 bits of the same network, and a falling divergence."""
from __future__ import annotations

import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qad():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import qad_step
    return qad_step


class Straight(torch.autograd.Function):
    """x replaced by its quantized value; the gradient passes as it is."""

    @staticmethod
    def forward(ctx, x, q):
        return q.double()

    @staticmethod
    def backward(ctx, g):
        return g, None


def reference(p, s, x, target, weight):
    """The student's network in 64 bits on the quantized values that the step used."""
    v = {k: t.double().cpu().requires_grad_() for k, t in p.items()}
    q = {k: Straight.apply(v[k], s["w"][k].cpu()) for k in ("w1", "w2", "w3")}
    x = x.double().cpu().requires_grad_()

    def norm(h, w, b, center):
        d = h - h.mean(-1, keepdim=True) if center else h
        return d * (d.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w + b
    q1 = Straight.apply(norm(x, v["n1"], v["b1"], True), s["q1"].cpu())
    h = x + (q1 @ q["w1"].t()).relu() @ q["w2"].t()
    q2 = Straight.apply(norm(h, v["n2"], 0.0, False), s["q2"].cpu())
    logits = q2 @ q["w3"].t()
    lp = torch.log_softmax(target.double().cpu(), 1)
    loss = (weight.double().cpu() * (lp.exp() * (lp - torch.log_softmax(logits, 1))).sum(1)).sum()
    loss.backward()
    return loss.item(), {**{k: t.grad for k, t in v.items()}, "x": x.grad}


def test_step_gradients(qad):
    """Every product's result and every gradient is rounded to bf16 once (2^-8 relative), and a
    gradient passes through at most eight such roundings on its way; they add up to at most
    8 * 2^-8 = 3.2 % of a tensor's norm."""
    nv = qad.nv
    teacher = qad.make_model(128, 256, 1000)
    student = qad.Student(teacher)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(96, 128, generator=gen, device="cuda").to(torch.bfloat16)
    weight = (torch.rand(96, generator=gen, device="cuda") < 0.7).float()
    target = qad.forward(teacher, teacher, x, quantize=False)["logits"]
    s = qad.forward(student.p, student.quantized(), x, quantize=True)
    for k in qad.MATRICES:                # the maxima that came along give the dynamic call's bits
        assert torch.equal(s["w"][k], nv.fakequant(student.p[k], qad.MODE, qad.RULE)[0])
    loss, dlogits = nv.distill_loss(s["logits"], target, weight)
    got = qad.backward(student.p, s, dlogits)
    want_loss, want = reference(student.p, s, x, target, weight)
    assert abs(loss.double().sum().item() - want_loss) <= 0.032 * want_loss
    for k, g in got.items():
        off = (g.double().cpu() - want[k]).norm() / want[k].norm()
        assert off <= 0.032, (k, float(off))


def test_divergence_falls(qad):
    losses = qad.main(tokens=512, width=256, hidden=512, vocab=2000, steps=30, lr=5e-4)
    assert all(v == v and v > 0 for v in losses)
    assert sum(losses[-5:]) < 0.8 * sum(losses[:5]), losses


def test_maxima_follow_the_weights(qad):
    teacher = qad.make_model(64, 128, 500)
    student = qad.Student(teacher)
    x = torch.randn(32, 64, device="cuda").to(torch.bfloat16)
    for _ in range(3):
        qad.step(student, teacher, x, torch.ones(32, device="cuda"), 1e-2)
        for i, k in enumerate(student.names):
            assert student.amax[i].item() == student.p[k].float().abs().max().item()
