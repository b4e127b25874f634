"""Quantization-aware distillation of a small two-layer student, with the package's operators.

A teacher in bf16 and a student whose weights and activations run through the NVFP4 fake-quant
("Quantization-Aware Distillation for NVFP4 Inference Accuracy Recovery", method section): per
step

    y1 = layer_norm(x)                    its maximum comes with it, so that
    q1 = fakequant(y1)                    reads y1 once
    h  = x + relu(q1 W1^T) W2^T           inside the second layer norm
    q2 = fakequant(layer_norm(h))
    logits = q2 W3^T
    loss, d logits = distill_loss(logits, teacher's logits)
    ... back through both layer norms (straight through the fake-quants) ...
    AdamW on all tensors at once, 8-bit states, bf16 weights by stochastic rounding; it delivers the
    maximum of each new weight, with which the next step's fake-quant reads the weight once.

The matrix products are the library's.  Run on an MI355X:  python examples/qad_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_block_scaled_amax_amd as nv  # noqa: E402

MODE, RULE = "four_over_six", "mse"
MATRICES = ("w1", "w2", "w3")              # fake-quantized; the norms' vectors are not


def make_model(width: int, hidden: int, vocab: int, seed: int = 0, device: str = "cuda") -> dict:
    gen = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device=device)
    m = {"w1": r(hidden, width) * width ** -0.5, "w2": r(width, hidden) * hidden ** -0.5,
         "w3": r(vocab, width) * width ** -0.5, "n1": torch.ones(width, device=device),
         "b1": torch.zeros(width, device=device), "n2": torch.ones(width, device=device)}
    return {k: v.to(torch.bfloat16) for k, v in m.items()}


class Student:
    """The student's tensors, their optimizer plan, and the maxima of its matrices."""

    def __init__(self, model: dict):
        self.p = {k: v.clone() for k, v in model.items()}
        self.names = list(self.p)
        self.plan = nv.adamw_plan(self.p.values(), state="e4m3")
        self.amax = torch.empty(len(self.names), device=self.p["w1"].device)
        for k in MATRICES:
            i = self.names.index(k)
            nv.amax(self.p[k], out=self.amax[i:i + 1])
        self.steps = 0

    def quantized(self) -> dict:
        """The matrices as the forward sees them."""
        q = {}
        for k in MATRICES:
            i = self.names.index(k)
            q[k] = nv.fakequant_from_amax(self.p[k], self.amax[i:i + 1], MODE, RULE)[0]
        return q

    def update(self, grads: dict, lr: float) -> None:
        self.steps += 1
        nv.adamw_step(self.plan, [grads[k] for k in self.names], step=self.steps, lr=lr,
                      weight_decay=0.0, amax=self.amax, seed=17)


def forward(p: dict, w: dict, x: torch.Tensor, quantize: bool) -> dict:
    """All that the backward pass needs; quantize=False is the teacher's forward."""
    top = torch.empty(1, device=x.device)
    fq = lambda y: nv.fakequant_from_amax(y, top, MODE, RULE)[0] if quantize else y
    s = {"x": x, "w": w}
    y1, _, s["mean1"], s["rstd1"] = nv.layer_norm(x, p["n1"], p["b1"], amax=top)
    s["q1"] = fq(y1)
    s["u"] = s["q1"] @ w["w1"].t()
    s["a"] = s["u"].relu()
    y2, s["h"], _, s["rstd2"] = nv.layer_norm(s["a"] @ w["w2"].t(), p["n2"], residual=x, center=False,
                                              amax=top)
    s["q2"] = fq(y2)
    s["logits"] = s["q2"] @ w["w3"].t()
    return s


def backward(p: dict, s: dict, dlogits: torch.Tensor) -> dict:
    w, g = s["w"], {}
    g["w3"] = dlogits.t() @ s["q2"]
    dh, g["n2"], _ = nv.layer_norm_backward(dlogits @ w["w3"], s["h"], p["n2"], None, s["rstd2"],
                                            bias=False)
    g["w2"] = dh.t() @ s["a"]
    du = (dh @ w["w2"]) * (s["u"] > 0)
    g["w1"] = du.t() @ s["q1"]
    g["x"], g["n1"], g["b1"] = nv.layer_norm_backward(du @ w["w1"], s["x"], p["n1"], s["mean1"],
                                                      s["rstd1"], dres=dh)
    return g


def step(student: Student, teacher: dict, x: torch.Tensor, weight: torch.Tensor, lr: float):
    """One training step -> the sum of the rows' losses, on the GPU."""
    target = forward(teacher, teacher, x, quantize=False)["logits"]
    s = forward(student.p, student.quantized(), x, quantize=True)
    loss, dlogits = nv.distill_loss(s["logits"], target, weight, grad=s["logits"])
    student.update(backward(student.p, s, dlogits), lr)
    return loss.sum()


def main(tokens=2048, width=1024, hidden=4096, vocab=32000, steps=20, lr=5e-4):
    """A student that starts some way off its teacher (its matrices 30 % noise) comes back."""
    teacher, noise = make_model(width, hidden, vocab), make_model(width, hidden, vocab, seed=2)
    student = Student({k: t + 0.3 * noise[k] if k in MATRICES else t for k, t in teacher.items()})
    gen = torch.Generator(device="cuda").manual_seed(1)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=gen, device="cuda").to(torch.bfloat16)
        weight = (torch.rand(tokens, generator=gen, device="cuda") < 0.8).float()   # answers only
        weight /= weight.sum()
        losses.append(step(student, teacher, x, weight, lr))
    losses = [float(v) for v in losses]
    print("divergence from the teacher, first and last step: %.5f %.5f" % (losses[0], losses[-1]))
    return losses


if __name__ == "__main__":
    main()
