"""The operators of a training step on a model's own answers: products of a few rows with packed
NVFP4 weights, log probabilities of given tokens forward and backward, the gradient norm and clipping.

A thin binding over ``libnvfp4_amax.so`` (``include/nvfp4_answer.h`` defines the operations), as
``train.py`` is: torch provides memory and the current stream, every step of the computation runs in
the library's kernels, and no call records an autograd graph.

    codes, scales, alpha = quantize(weight)                      # packed once
    y = packed_matvec(x, codes, scales, alpha)                   # the next token's products
    logp, entropy, top_logp, top_index, stats = token_logprobs(logits, tokens, top=20)
    dlogits = token_logprobs_backward(logits, tokens, stats, dlogp)
    norm, scale = grad_norm(plan, grads, max_norm=1.0)
    adamw_step(plan, grads, step=1, lr=1e-4, grad_scale=scale)   # or clip_grads(plan, grads, scale)
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import lib
from .train import (_BOTH, _F32, TYPES, AdamWPlan, _call, _like, _out, _ptr, _rows, _type, _vector,
                    _work)

INDICES = {torch.int32: 0, torch.int64: 1}
_U8 = (torch.uint8,)
ANSWER_ABI_VERSION = 1          # NVFP4_ANSWER_ABI_VERSION
MATVEC_MAX_ROWS = 1024          # NVFP4_MATVEC_MAX_ROWS
LOGPROBS_MAX = 64               # NVFP4_LOGPROBS_MAX


def grad_norm_workspace(count: int) -> int:
    """NVFP4_GRAD_NORM_WORKSPACE(count): bytes of grad_norm's workspace for `count` tensors."""
    return 16384 * (count // 200 + 1)


def bind(L: ctypes.CDLL) -> None:
    """Argument types of the entry points of nvfp4_answer.h."""
    P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    f32, f64 = ctypes.c_float, ctypes.c_double
    L.nvfp4_answer_abi_version.restype = i32
    if L.nvfp4_answer_abi_version() != ANSWER_ABI_VERSION:
        raise RuntimeError("libnvfp4_amax.so has answer ABI version %d, this binding needs %d: "
                           "rebuild it" % (L.nvfp4_answer_abi_version(), ANSWER_ABI_VERSION))
    L.nvfp4_packed_matvec.argtypes = [P, i64, P, P, P, P, i64, i64, i64, i64, i64, i32, i32, i32, P, P]
    L.nvfp4_token_logprobs_workspace.argtypes = [i64, i64, i64]
    L.nvfp4_token_logprobs_workspace.restype = i64
    L.nvfp4_token_logprobs.argtypes = [P, i64, P, i64, i64, i64, i64, i32, i32, f32, P, P, P, P, P, P, P]
    L.nvfp4_token_logprobs_backward.argtypes = [P, i64, P, P, P, P, P, i64, i64, i64, i32, i32, f32, P,
                                                i64, P]
    L.nvfp4_grad_norm.argtypes = [P, i64, i32, f64, f64, P, P, P, P]
    L.nvfp4_clip_grads.argtypes = [P, P, i64, i32, P, P]
    for name in ("nvfp4_packed_matvec", "nvfp4_token_logprobs", "nvfp4_token_logprobs_backward",
                 "nvfp4_grad_norm", "nvfp4_clip_grads"):
        getattr(L, name).restype = i32


def _output(t, shape, dtype, x: torch.Tensor) -> torch.Tensor:
    """The caller's output, checked, or a new one.  (Sizes one by one: torch takes 1.1 us for these and 1.6
    for a tuple, and a call has up to five outputs.)"""
    if t is None and shape:
        return x.new_empty(*shape, dtype=dtype)
    return _out(t, shape, dtype, x)


def packed_matvec(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, alpha: torch.Tensor, *,
                  expert: torch.Tensor = None, dtype: torch.dtype = None, y=None):
    """x W^T for a few rows of x with a packed NVFP4 weight -> y [..., rows].

    x is [..., cols], bfloat16 or float32 (2-D with a row stride, or contiguous); codes, scales and alpha
    as quantize returns them for a [rows, cols] weight.  With expert they are those of a [E, rows, cols]
    batch: x is [tokens, cols], expert int32 or int64 [tokens] or [tokens, picks], and y [tokens, rows] or
    [tokens, picks, rows] holds each token's product with the weight of each of its experts (zeros for
    an index outside 0 .. E - 1).  dtype: y's, bfloat16 or float32 (default: x's).  At most
    MATVEC_MAX_ROWS rows of y: a product of more is one for dequantize and a matrix product."""
    shape = x.shape
    xs, kind = _rows(x, shape, "x"), _type(x, "x")
    cols = shape[-1]
    lead = codes.dim() - 2
    if lead != (0 if expert is None else 1):
        raise ValueError("codes must be [rows, cols/2], or [E, rows, cols/2] with expert")
    if cols % 16:
        raise ValueError("x must have a last dimension that is a multiple of 16")
    E, rows = (1 if expert is None else codes.shape[0]), codes.shape[lead]
    head = (E, rows) if lead else (rows,)
    _vector(codes, (*head, cols // 2), _U8, x, "codes")
    _vector(scales, (*head, cols // 16), _U8, x, "scales")
    _vector(alpha, (E,), _F32, x, "alpha")
    tokens, picks, itype = x.numel() // cols, 1, 0
    to = shape[:-1]
    if expert is not None:
        if len(shape) != 2:
            raise ValueError("x must be [tokens, cols] with expert")
        to = expert.shape
        if len(to) not in (1, 2) or to[0] != tokens:
            raise ValueError("expert must be [tokens] or [tokens, picks]")
        _vector(expert, to, tuple(INDICES), x, "expert")
        itype = INDICES[expert.dtype]
        picks = to[1] if len(to) == 2 else 1
    if tokens * picks > MATVEC_MAX_ROWS:
        raise ValueError("at most %d rows, got %d" % (MATVEC_MAX_ROWS, tokens * picks))
    dtype = x.dtype if dtype is None else dtype
    if dtype not in TYPES:
        raise TypeError("dtype must be bfloat16 or float32, got %s" % dtype)
    y = _output(y, (*to, rows), dtype, x)
    if y.numel() == 0:
        return y
    _call("nvfp4_packed_matvec", x, x.data_ptr(), xs, codes.data_ptr(), scales.data_ptr(),
          alpha.data_ptr(), _ptr(expert), tokens, picks, E, rows, cols, kind, TYPES[dtype], itype,
          y.data_ptr())
    return y


def _given(tokens: torch.Tensor, lead, x: torch.Tensor) -> int:
    """How many tokens a row has: tokens is [...] or [..., given]."""
    if tokens.shape[:len(lead)] != lead or tokens.dim() > len(lead) + 1:
        raise ValueError("tokens must have shape %s or %s + [given], got %s"
                         % (tuple(lead), tuple(lead), tuple(tokens.shape)))
    _vector(tokens, tokens.shape, tuple(INDICES), x, "tokens")
    given = tokens.shape[-1] if tokens.dim() > len(lead) else 1
    if not 1 <= given <= LOGPROBS_MAX:
        raise ValueError("1 to %d tokens a row, got %d" % (LOGPROBS_MAX, given))
    return given


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor = None, *, top: int = 0,
                   temperature: float = 1.0, logp=None, entropy=None, top_logp=None, top_index=None,
                   stats=None, workspace=None):
    """Log probabilities of given tokens under softmax(logits / temperature)
    -> (logp, entropy, top_logp, top_index, stats).

    logits is [..., vocab], bfloat16 or float32, contiguous; 2-D ones may have a row stride.  (The
    logits[:, :-1] of a batch are neither: pass all of them, with -1 for each last token.)  tokens: int32 or
    int64, [...] (one a row) or [..., given]; logp has their shape.  A token of -1 is none (logp 0), and
    rows that have none but these are not read (zeros; top_index -1).  entropy is [...], in nats.  top:
    how many of the largest entries to return, in falling order, the lowest index first among equals:
    top_logp and top_index (int64) are [..., top], or None.  stats [..., 2] (the largest logit, and
    ln sum exp((x - largest) / temperature)) is for the backward pass.  Without tokens logp is None.
    Outside of autograd: token_logprobs_backward is the gradient."""
    shape = logits.shape
    xs, kind = _rows(logits, shape, "logits"), _type(logits, "logits")
    lead, vocab = shape[:-1], shape[-1]
    if not 0 <= top <= min(LOGPROBS_MAX, vocab):
        raise ValueError("top must be in 0 .. %d, got %d" % (min(LOGPROBS_MAX, vocab), top))
    given, itype = 0, 0
    if tokens is not None:
        given, itype = _given(tokens, lead, logits), INDICES[tokens.dtype]
        logp = _output(logp, tokens.shape, torch.float32, logits)
    elif logp is not None:
        raise ValueError("logp is an output of the form with tokens only")
    entropy = _output(entropy, lead, torch.float32, logits)
    stats = _output(stats, (*lead, 2), torch.float32, logits)
    if top:
        top_logp = _output(top_logp, (*lead, top), torch.float32, logits)
        top_index = _output(top_index, (*lead, top), torch.int64, logits)
    elif top_logp is not None or top_index is not None:
        raise ValueError("top_logp and top_index are outputs of the form with top only")
    rows = entropy.numel()
    need = lib().nvfp4_token_logprobs_workspace(rows, vocab, top)
    ws = _work(workspace, need, logits) if need else None
    _call("nvfp4_token_logprobs", logits, logits.data_ptr(), xs, _ptr(tokens), rows, vocab, given, top,
          kind, itype, temperature, _ptr(logp), entropy.data_ptr(), _ptr(top_logp), _ptr(top_index),
          stats.data_ptr(), _ptr(ws))
    return logp, entropy, top_logp, top_index, stats


def token_logprobs_backward(logits: torch.Tensor, tokens: torch.Tensor, stats: torch.Tensor,
                            dlogp: torch.Tensor, *, entropy: torch.Tensor = None,
                            dentropy: torch.Tensor = None, temperature: float = 1.0, grad=None):
    """Gradient of token_logprobs with respect to the logits -> grad in logits' type.

    tokens, stats, entropy and temperature as in the forward call; dlogp float32 in tokens' shape;
    dentropy float32 [...] (with entropy) or None.  Rows without a token have a gradient of 0; equal tokens of
    a row add up.  grad may be logits itself (written in place)."""
    shape = logits.shape
    xs, kind = _rows(logits, shape, "logits"), _type(logits, "logits")
    lead, vocab = shape[:-1], shape[-1]
    given = _given(tokens, lead, logits)
    _vector(stats, lead + (2,), _F32, logits, "stats")
    _vector(dlogp, tokens.shape, _F32, logits, "dlogp")
    if dentropy is not None:
        if entropy is None:
            raise ValueError("dentropy needs entropy")
        _vector(dentropy, lead, _F32, logits, "dentropy")
        _vector(entropy, lead, _F32, logits, "entropy")
    gs = vocab
    if grad is not None:
        _like(grad, shape, (logits.dtype,), logits, "grad")
        gs = _rows(grad, shape, "grad")
    else:
        grad = torch.empty_like(logits) if xs == vocab else _out(None, shape, logits.dtype, logits)
    rows = stats.numel() // 2
    _call("nvfp4_token_logprobs_backward", logits, logits.data_ptr(), xs, tokens.data_ptr(),
          stats.data_ptr(), _ptr(entropy) if dentropy is not None else None, dlogp.data_ptr(),
          _ptr(dentropy), rows, vocab, given, kind, INDICES[tokens.dtype], temperature, grad.data_ptr(), gs)
    return grad


def _table(plan: AdamWPlan, grads) -> bytes:
    """The entries of nvfp4_grad_tensor for these tensors.  (Packed at once: half the time of an array of
    numpy's, and of each call its own.)"""
    entries = [0] * (2 * len(grads))
    entries[0::2] = map(torch.Tensor.data_ptr, grads)
    entries[1::2] = plan.numels
    return struct.pack("%dq" % len(entries), *entries)


def _look(plan: AdamWPlan, grads):
    grads = list(grads)
    if len(grads) != len(plan.params):
        raise ValueError("%d gradients for %d parameters" % (len(grads), len(plan.params)))
    return grads, plan._look_grads(grads)


def grad_norm(plan: AdamWPlan, grads, *, max_norm: float = None, eps: float = 1e-6, norm=None, scale=None,
              workspace=None):
    """The 2-norm over all elements of a plan's gradients -> (norm, scale), float32 [1] on the GPU.

    scale = min(1, max_norm / (norm + eps)) is what adamw_step takes as grad_scale and clip_grads
    multiplies by; None without max_norm.  Nothing waits for the GPU.  Gradients as in adamw_step."""
    grads, kind = _look(plan, grads)
    like = plan.params[0]
    norm = _output(norm, (1,), torch.float32, like)
    if max_norm is not None:
        scale = _output(scale, (1,), torch.float32, like)
    elif scale is not None:
        raise ValueError("scale is an output of the form with max_norm only")
    ws = _work(workspace, grad_norm_workspace(len(grads)), like)
    _call("nvfp4_grad_norm", like, _table(plan, grads), len(grads), kind,
          0.0 if max_norm is None else max_norm, eps, norm.data_ptr(), _ptr(scale), ws.data_ptr())
    return norm, scale


def clip_grads(plan: AdamWPlan, grads, scale: torch.Tensor, *, out=None):
    """Gradients times scale (float32 [1] on the GPU, from grad_norm) -> the list of them.

    In place, where a scale of 1 leaves them alone, or into out: one tensor per gradient, like it.
    adamw_step(grad_scale=scale) does the same on its way, without a pass over the gradients."""
    grads, kind = _look(plan, grads)
    like = plan.params[0]
    _vector(scale, (1,), _F32, like, "scale")
    to = None
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError("%d outputs for %d gradients" % (len(out), len(grads)))
        # (those that were checked were all of one type, which need not be that of these gradients)
        if not (out and out[0].dtype == grads[0].dtype and plan._seen_out.again(out)):
            for t, n in zip(out, plan.numels):
                plan._look("out", t, n, grads[0].dtype)
            plan._seen_out.keep(out)
        to = _table(plan, out)
    _call("nvfp4_clip_grads", like, _table(plan, grads), to, len(grads), kind, scale.data_ptr())
    return grads if out is None else out
