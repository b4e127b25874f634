"""A training step on the student's own answers, with the package's operators.

The student of qad_step.py, its weights packed, draws tokens; its teacher and it score them; and
the student is moved towards tokens that the teacher finds likelier than it does (on-policy
distillation: the gradient of D_KL(p_student || p_teacher) along the student's own answers,
estimated by its tokens' log probabilities, with an entropy bonus):

    answers   packed_matvec with codes, scales and alpha of each matrix, a token at a time for all
              answers; token_logprobs' alternatives to draw the next one from
    scores    token_logprobs of the drawn tokens, under both models
    gradient  token_logprobs_backward, then back through the network as in qad_step.py
    update    grad_norm and adamw_step, which takes the clipping coefficient on its way

Weights are 4-bit in the answers and fake-quantized in the training pass (W4A16): both see the same values.
Run on an MI355X:  python examples/answer_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import qad_step as qad  # noqa: E402
from qad_step import nv  # noqa: E402

ALTERNATIVES = 20                          # tokens that the next one is drawn from
BONUS = 0.01                               # weight of the entropy
MAX_NORM = 1.0


def pack(student: qad.Student) -> dict:
    """The student's matrices as codes, scales and alpha, from the maxima that came with its last update."""
    packed = {}
    for k in qad.MATRICES:
        i = student.names.index(k)
        packed[k] = nv.quantize_from_amax(student.p[k], student.amax[i:i + 1], qad.MODE, qad.RULE)
    return packed


def answer_logits(p: dict, packed: dict, x: torch.Tensor) -> torch.Tensor:
    """qad_step.forward without fake-quantized activations, for a few rows and packed weights."""
    y1 = nv.layer_norm(x, p["n1"], p["b1"])[0]
    a = nv.packed_matvec(y1, *packed["w1"]).relu_()
    y2 = nv.layer_norm(nv.packed_matvec(a, *packed["w2"]), p["n2"], residual=x, center=False)[0]
    return nv.packed_matvec(y2, *packed["w3"], dtype=torch.float32)


def draw(p: dict, packed: dict, embed: torch.Tensor, x: torch.Tensor, length: int, gen: torch.Generator):
    """Answers of `length` tokens to the rows of x -> (inputs [length * rows, width], tokens [length * rows])."""
    inputs, tokens = [], []
    for _ in range(length):
        inputs.append(x)
        logits = answer_logits(p, packed, x)
        _, _, top_logp, top_index, _ = nv.token_logprobs(logits, top=ALTERNATIVES)
        noise = torch.rand(top_logp.shape, generator=gen, device=x.device)
        pick = (top_logp - (-noise.log()).log()).argmax(1, keepdim=True)      # one of them, by its probability
        tokens.append(top_index.gather(1, pick)[:, 0])
        x = embed[tokens[-1]]
    return torch.cat(inputs), torch.cat(tokens)


def gradients(student: qad.Student, teacher: dict, x: torch.Tensor, tokens: torch.Tensor):
    """-> (gradients by name, log probability under the student minus that under the teacher, per token)."""
    target = qad.forward(teacher, teacher, x, quantize=False)["logits"]
    s = qad.forward(student.p, student.quantized(), x, quantize=False)
    logp, entropy, _, _, stats = nv.token_logprobs(s["logits"], tokens)
    ahead = logp - nv.token_logprobs(target, tokens)[0]
    # of mean(ahead * logp) - BONUS * mean(entropy), ahead held
    scale = 1.0 / tokens.numel()
    dlogits = nv.token_logprobs_backward(s["logits"], tokens, stats, ahead * scale, entropy=entropy,
                                         dentropy=torch.full_like(entropy, -BONUS * scale), grad=s["logits"])
    return qad.backward(student.p, s, dlogits), ahead


def step(student: qad.Student, teacher: dict, embed: torch.Tensor, x: torch.Tensor, length: int, lr: float,
         gen: torch.Generator):
    """One training step -> (how far the student is ahead of its teacher on its own tokens, the gradient's norm)."""
    inputs, tokens = draw(student.p, pack(student), embed, x, length, gen)
    grads, ahead = gradients(student, teacher, inputs, tokens)
    listed = [grads[k] for k in student.names]
    norm, scale = nv.grad_norm(student.plan, listed, max_norm=MAX_NORM)
    student.steps += 1
    nv.adamw_step(student.plan, listed, step=student.steps, lr=lr, weight_decay=0.0, grad_scale=scale,
                  amax=student.amax, seed=17)
    return ahead.mean(), norm


def main(answers=16, length=32, width=1024, hidden=4096, vocab=32000, steps=20, lr=1e-4):
    teacher, noise = qad.make_model(width, hidden, vocab), qad.make_model(width, hidden, vocab, seed=2)
    student = qad.Student({k: t + 0.3 * noise[k] if k in qad.MATRICES else t for k, t in teacher.items()})
    gen = torch.Generator(device="cuda").manual_seed(1)
    embed = torch.randn(vocab, width, generator=gen, device="cuda").to(torch.bfloat16)
    got = []
    for _ in range(steps):
        x = embed[torch.randint(vocab, (answers,), generator=gen, device="cuda")]
        got.append(step(student, teacher, embed, x, length, lr, gen))
    got = [(float(a), float(n)) for a, n in got]
    print("student ahead of its teacher on its own tokens, first and last step: %.4f %.4f" % (got[0][0], got[-1][0]))
    return got


if __name__ == "__main__":
    main()
