"""The step on the student's own answers of examples/answer_step.py: its packed answers against the
fake-quantized network, its gradients against automatic differentiation in 64 bits, and that it runs."""
from __future__ import annotations

import math
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ans():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import answer_step
    return answer_step


def norm(h, w, b, center):
    d = h - h.mean(-1, keepdim=True) if center else h
    return d * (d.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * w + b


def student_of(ans, width, hidden, vocab):
    teacher, noise = ans.qad.make_model(width, hidden, vocab), ans.qad.make_model(width, hidden, vocab, seed=2)
    return teacher, ans.qad.Student({k: t + 0.3 * noise[k] if k in ans.qad.MATRICES else t
                                     for k, t in teacher.items()})


@pytest.mark.parametrize("rows", [1, 5, 16, 40])
@pytest.mark.parametrize("width,hidden,vocab", [(128, 272, 1000), (1040, 2064, 3001)])
def test_packed_answers(ans, rows, width, hidden, vocab):
    """The logits of packed weights are those of the fake-quantized ones: both differ from the
    exact network by one bf16 rounding per product, norm and weight, of which a value passes at most eight
    (2^-9 each, 2^-8 with both networks' errors), as a share of the logits' norm."""
    _, student = student_of(ans, width, hidden, vocab)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, width, generator=gen, device="cuda").to(torch.bfloat16)
    got = ans.answer_logits(student.p, ans.pack(student), x)
    want = ans.qad.forward(student.p, student.quantized(), x, quantize=False)["logits"]
    assert (got - want.float()).norm() <= 8 * 2.0 ** -8 * want.float().norm()


def test_drawn_tokens_are_among_the_alternatives(ans):
    nv = ans.nv
    _, student = student_of(ans, 128, 256, 1000)
    gen = torch.Generator(device="cuda").manual_seed(3)
    embed = torch.randn(1000, 128, generator=gen, device="cuda").to(torch.bfloat16)
    packed = ans.pack(student)
    inputs, tokens = ans.draw(student.p, packed, embed, embed[:7], 5, gen)
    assert inputs.shape == (35, 128) and tokens.shape == (35,)
    assert torch.equal(inputs[7:], embed[tokens[:28]])
    for i in range(0, 35, 7):                 # the products of the same rows: the same bits
        logits = ans.answer_logits(student.p, packed, inputs[i:i + 7])
        top = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :ans.ALTERNATIVES]
        assert (top == tokens[i:i + 7, None]).any(1).all()
        assert torch.equal(nv.token_logprobs(logits, top=ans.ALTERNATIVES)[3], top)


def test_gradients(ans):
    """Every product's result and every gradient is rounded to bf16 once (2^-8 relative), and a gradient
    passes through at most eight such roundings on its way: at most 8 * 2^-8 = 3.2 % of a tensor's norm.  What the
    tokens' scores are off by is a rounding of the logits too (2^-8 of their size) and enters as a ninth."""
    teacher, student = student_of(ans, 128, 256, 1000)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(96, 128, generator=gen, device="cuda").to(torch.bfloat16)
    tokens = torch.randint(1000, (96,), generator=gen, device="cuda")
    q = {k: w.double().cpu() for k, w in student.quantized().items()}
    got, ahead = ans.gradients(student, teacher, x, tokens)
    v = {k: t.double().cpu().requires_grad_() for k, t in student.p.items()}
    w = {k: q[k] + v[k] - v[k].detach() for k in q}              # straight through
    xs = x.double().cpu().requires_grad_()
    h = xs + (norm(xs, v["n1"], v["b1"], True) @ w["w1"].t()).relu() @ w["w2"].t()
    lp = torch.log_softmax(norm(h, v["n2"], 0.0, False) @ w["w3"].t(), 1)
    logp = lp.gather(1, tokens.cpu()[:, None])[:, 0]
    entropy = -(lp.exp() * lp).sum(1)
    ((ahead.double().cpu() * logp).mean() - ans.BONUS * entropy.mean()).backward()
    want = {**{k: t.grad for k, t in v.items()}, "x": xs.grad}
    for k, g in got.items():
        off = (g.double().cpu() - want[k]).norm() / want[k].norm()
        assert off <= 9 * 2.0 ** -8, (k, float(off))


def test_it_runs(ans):
    got = ans.main(answers=5, length=4, width=256, hidden=512, vocab=2000, steps=4)
    assert len(got) == 4 and all(math.isfinite(a) and math.isfinite(n) and n > 0 for a, n in got)


def test_the_update_is_clipped(ans):
    """The step moves the weights as one on gradients scaled to the norm allowed, bit for bit in the states'
    own arithmetic: the coefficient multiplies each gradient in 32 bits either way."""
    nv = ans.nv
    teacher, student = student_of(ans, 64, 128, 500)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(32, 64, generator=gen, device="cuda").to(torch.bfloat16)
    tokens = torch.randint(500, (32,), generator=gen, device="cuda")
    grads = [ans.gradients(student, teacher, x, tokens)[0][k].float() for k in student.names]
    params = [student.p[k].clone() for k in student.names]
    norm_, scale = nv.grad_norm(student.plan, grads, max_norm=1e-3)
    total = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(norm_.item() - total) <= 2.0 ** -23 * total and scale.item() < 1
    nv.adamw_step(student.plan, grads, step=1, lr=1e-3, grad_scale=scale, seed=9)
    other = nv.adamw_plan(params, state="e4m3")
    nv.adamw_step(other, nv.clip_grads(other, grads, scale), step=1, lr=1e-3, seed=9)
    for a, b in zip(student.plan.params + student.plan.exp_avg, other.params + other.exp_avg):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
