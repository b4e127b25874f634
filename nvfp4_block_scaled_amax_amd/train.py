"""The operators of a quantization-aware distillation step around fake-quantization: layer norm
forward and backward, the distillation loss with its gradient, AdamW over many tensors.

A thin binding over ``libnvfp4_amax.so`` (``include/nvfp4_train.h`` defines the operations).
As in the quantization calls, torch provides memory and the current stream and every step of the
computation runs in the library's kernels.

    y, h, mean, rstd = layer_norm(x, weight, bias, residual=r, amax=top)   # h = x + r
    q, _ = fakequant_from_amax(y, top, ...)                                # no amax pass over y
    loss, grad = distill_loss(student_logits, teacher_logits, row_weight)
    dx, dweight, dbias = layer_norm_backward(dy, h, weight, mean, rstd, dres=dh)
    plan = adamw_plan(params, state="e4m3")
    adamw_step(plan, grads, step=1, lr=1e-4, seed=0)

Tensors are bfloat16 or float32, on one GPU, with a contiguous last dimension.  No call records
an autograd graph, whatever `requires_grad` says: results have none, and a training loop passes
the gradients on itself (examples/qad_step.py) or from a torch.autograd.Function of its own.
"""
from __future__ import annotations

import ctypes
from itertools import chain

import numpy as np
import torch

from . import NVFP4Error, lib

TYPES = {torch.bfloat16: 0, torch.float32: 1}
STATES = {"f32": 0, "e4m3": 1}
ADAMW_BLOCK = 128               # NVFP4_ADAMW_BLOCK: elements per scale of an 8-bit state
TRAIN_ABI_VERSION = 1           # NVFP4_TRAIN_ABI_VERSION


class AdamWTensor(ctypes.Structure):
    """nvfp4_adamw_tensor."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "exp_avg", "exp_avg_sq", "master",
                                               "avg_scale", "sq_scale")] + [("numel", ctypes.c_int64)]


class AdamWArgs(ctypes.Structure):
    """nvfp4_adamw_args."""
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [
        ("step", ctypes.c_int64), ("seed", ctypes.c_uint32)]


def bind(L: ctypes.CDLL) -> None:
    """Argument types of the entry points of nvfp4_train.h."""
    P, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    L.nvfp4_train_abi_version.restype = i32
    if L.nvfp4_train_abi_version() != TRAIN_ABI_VERSION:
        raise RuntimeError("libnvfp4_amax.so has training ABI version %d, this binding needs %d: "
                           "rebuild it" % (L.nvfp4_train_abi_version(), TRAIN_ABI_VERSION))
    L.nvfp4_train_status_str.argtypes, L.nvfp4_train_status_str.restype = [i32], ctypes.c_char_p
    L.nvfp4_layernorm_forward.argtypes = [P, i64, P, i64, P, P, i64, i64, i32, i32, i32, f32, P, P,
                                          P, P, P, P]
    L.nvfp4_layernorm_backward_workspace.argtypes = [i64, i64]
    L.nvfp4_layernorm_backward_workspace.restype = i64
    L.nvfp4_layernorm_backward.argtypes = [P, P, P, P, P, P, i64, i64, i32, i32, P, P, P, P, P]
    L.nvfp4_distill_loss_workspace.argtypes = [i64, i64]
    L.nvfp4_distill_loss_workspace.restype = i64
    L.nvfp4_distill_loss.argtypes = [P, i64, P, i64, P, i64, i64, i32, i32, f32, P, P, i64, P, P]
    L.nvfp4_adamw_step.argtypes = [P, i64, i32, i32, i32, P, P, P, P]
    for name in ("nvfp4_layernorm_forward", "nvfp4_layernorm_backward", "nvfp4_distill_loss",
                 "nvfp4_adamw_step"):
        getattr(L, name).restype = i32


def _call(name: str, x: torch.Tensor, *args):
    """The entry point `name` on x's device and its current stream; raises on an error status.
    (A call of a few microseconds: the device is only switched where it has to be.)"""
    fn, dev = getattr(lib(), name), x.get_device()
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status != 0:
        raise NVFP4Error(status, name, lib().nvfp4_train_status_str(status).decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _type(t: torch.Tensor, what: str) -> int:
    kind = TYPES.get(t.dtype)
    if kind is None:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (what, t.dtype))
    return kind


def _rows(t: torch.Tensor, shape, what: str) -> int:
    """The row stride of a tensor seen as rows of its last dimension."""
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % what)
    if len(shape) == 0 or shape[-1] < 1:
        raise ValueError("%s must have a last dimension of at least 1" % what)
    if t.is_contiguous():
        return shape[-1]
    if len(shape) == 2 and (t.stride(1) == 1 or shape[1] == 1) and t.stride(0) >= shape[1]:
        return t.stride(0)
    raise ValueError("%s must be contiguous, or 2-D with a contiguous last dimension and rows "
                     "that do not overlap" % what)


def _like(t: torch.Tensor, shape, dtypes, x: torch.Tensor, what: str):
    """Checks a tensor that goes with x: its shape, its type, its device."""
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (what, " or ".join(map(str, dtypes)), t.dtype))
    if t.get_device() != x.get_device():
        raise ValueError("%s must be on %s" % (what, x.device))


def _vector(t: torch.Tensor, shape, dtypes, x: torch.Tensor, what: str):
    """The same, and that it is contiguous.  (One condition: it is what small calls wait for.)"""
    if not (t.shape == shape and t.dtype in dtypes and t.is_contiguous()
            and t.get_device() == x.get_device()):
        _like(t, shape, dtypes, x, what)
        raise ValueError("%s must be contiguous" % what)


def _out(t, shape, dtype, x: torch.Tensor) -> torch.Tensor:
    """The caller's output, checked, or a new one.  (The callers make those that are like a contiguous
    tensor with torch.empty_like, in two thirds of the time.)"""
    if t is None:
        return x.new_empty(shape, dtype=dtype)
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.device != x.device:
        raise ValueError("output must be a contiguous %s tensor of shape %s on %s"
                         % (dtype, tuple(shape), x.device))
    return t


def _work(workspace, nbytes: int, x: torch.Tensor):
    """The caller's workspace, checked, or one of `nbytes` bytes."""
    if nbytes < 0:
        raise ValueError("bad shape")
    if workspace is None:
        return x.new_empty(nbytes, dtype=torch.uint8)
    if (workspace.device != x.device or not workspace.is_contiguous()
            or workspace.numel() * workspace.element_size() < nbytes):
        raise ValueError("workspace must be a contiguous tensor of at least %d bytes on %s"
                         % (nbytes, x.device))
    return workspace


_F32 = (torch.float32,)
_BOTH = (torch.bfloat16, torch.float32)


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor = None, *,
               residual: torch.Tensor = None, eps: float = 1e-5, center: bool = True,
               amax: torch.Tensor = None, y=None, h=None, mean=None, rstd=None):
    """Layer norm of the last dimension -> (y, h, mean, rstd).

    h = x + residual rounded to x's type (x itself without residual); y = (h - mean) * rstd *
    weight + bias.  center=False is the root-mean-square norm (mean is None).  mean and rstd
    are float32, one per row, for the backward pass.  amax: float32 [1], receives max |y| for
    fakequant_from_amax / quantize_from_amax.  x and residual may be 2-D with a row stride.
    y may be x (without residual) and h may be x or residual, where they are contiguous.
    Outside of autograd: layer_norm_backward is the gradient."""
    shape, dtype = x.shape, x.dtype
    xs, kind = _rows(x, shape, "x"), _type(x, "x")
    lead, cols = shape[:-1], shape[-1]
    _vector(weight, shape[-1:], _BOTH, x, "weight")
    if bias is not None:
        _vector(bias, shape[-1:], (weight.dtype,), x, "bias")
    rs = cols
    if residual is not None:
        _like(residual, shape, (dtype,), x, "residual")
        rs = _rows(residual, shape, "residual")
        h = torch.empty_like(x) if h is None and xs == cols else _out(h, shape, dtype, x)
    elif h is not None:
        raise ValueError("h is an output of the residual form only")
    y = torch.empty_like(x) if y is None and xs == cols else _out(y, shape, dtype, x)
    rstd = _out(rstd, lead, torch.float32, x)
    if center:
        mean = torch.empty_like(rstd) if mean is None else _out(mean, lead, torch.float32, x)
    else:
        mean = None
    if amax is not None:
        _vector(amax, (1,), _F32, x, "amax")
    _call("nvfp4_layernorm_forward", x, x.data_ptr(), xs, _ptr(residual), rs, weight.data_ptr(),
          _ptr(bias), rstd.numel(), cols, kind, TYPES[weight.dtype], int(center), eps, y.data_ptr(),
          _ptr(h), _ptr(mean), rstd.data_ptr(), _ptr(amax))
    return y, x if residual is None else h, mean, rstd


def layer_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                        mean: torch.Tensor, rstd: torch.Tensor, *, dres: torch.Tensor = None,
                        bias: bool = True, dx=None, dweight=None, dbias=None, workspace=None):
    """Gradient of layer_norm -> (dx, dweight, dbias).

    h, mean and rstd as layer_norm returned them (mean None for center=False).  dres: gradient
    that reaches h past the norm, added to dx.  dx is the gradient of x and of residual alike, and may
    be written over dy or dres.  bias=False leaves dbias out (None)."""
    shape, dtype = dy.shape, dy.dtype
    _rows(dy, shape, "dy")
    kind = _type(dy, "dy")
    lead, cols = shape[:-1], shape[-1]
    if not dy.is_contiguous():
        raise ValueError("dy must be contiguous")
    _vector(h, shape, (dtype,), dy, "h")
    if dres is not None:
        _vector(dres, shape, (dtype,), dy, "dres")
    _vector(weight, shape[-1:], _BOTH, dy, "weight")
    _vector(rstd, lead, _F32, dy, "rstd")
    if mean is not None:
        _vector(mean, lead, _F32, dy, "mean")
    rows, wtype = rstd.numel(), weight.dtype
    dx = torch.empty_like(dy) if dx is None else _out(dx, shape, dtype, dy)
    dweight = torch.empty_like(weight) if dweight is None else _out(dweight, shape[-1:], wtype, dy)
    if bias:
        dbias = torch.empty_like(weight) if dbias is None else _out(dbias, shape[-1:], wtype, dy)
    else:
        dbias = None
    ws = _work(workspace, lib().nvfp4_layernorm_backward_workspace(rows, cols), dy)
    _call("nvfp4_layernorm_backward", dy, dy.data_ptr(), h.data_ptr(), weight.data_ptr(), _ptr(mean),
          rstd.data_ptr(), _ptr(dres), rows, cols, kind, TYPES[wtype], dx.data_ptr(),
          dweight.data_ptr(), _ptr(dbias), ws.data_ptr())
    return dx, dweight, dbias


def distill_loss(student: torch.Tensor, teacher: torch.Tensor, weight: torch.Tensor = None, *,
                 temperature: float = 1.0, want_grad: bool = True, loss=None, grad=None,
                 workspace=None):
    """weight * KL(softmax(teacher / T) || softmax(student / T)) per row, and its gradient with
    respect to the student's logits -> (loss float32 [...], grad in student's type or None).

    Logits are [..., vocab]; 2-D ones may have a row stride.  weight: float32 [...]; rows of
    weight 0 are not read.  grad may be the student itself (written in place).  Outside of
    autograd: loss has no graph, grad is what goes back from it."""
    shape = student.shape
    ss, kind = _rows(student, shape, "student"), _type(student, "student")
    lead, vocab = shape[:-1], shape[-1]
    _like(teacher, shape, _BOTH, student, "teacher")
    ts = _rows(teacher, shape, "teacher")
    if weight is not None:
        _vector(weight, lead, _F32, student, "weight")
    if loss is None and weight is not None:
        loss = torch.empty_like(weight)
    else:
        loss = _out(loss, lead, torch.float32, student)
    gs = vocab
    if grad is not None:
        if not want_grad:
            raise ValueError("grad is an output of the form with a gradient only")
        _like(grad, shape, (student.dtype,), student, "grad")
        gs = _rows(grad, shape, "grad")
    elif want_grad:
        grad = torch.empty_like(student) if ss == vocab else _out(None, shape, student.dtype, student)
    rows = loss.numel()
    need = lib().nvfp4_distill_loss_workspace(rows, vocab)
    ws = _work(workspace, need, student) if need else None
    _call("nvfp4_distill_loss", student, student.data_ptr(), ss, teacher.data_ptr(), ts, _ptr(weight),
          rows, vocab, kind, TYPES[teacher.dtype], temperature, loss.data_ptr(), _ptr(grad), gs,
          _ptr(ws))
    return loss, grad


class _Seen:
    """Tensors that were checked, to be recognized at the next step: the same sizes, strides, types and
    devices in the same order.  (An address does not tell: a view of a tensor, and what is put into its
    freed memory, begin where it did.)  torch compares a whole list in one call, 3 us for 72 tensors, where
    their attributes take 11 one by one; what it does not recognize is checked again in full."""

    def __init__(self):
        self._guards = None

    def keep(self, tensors) -> None:
        try:
            self._guards = torch._C._dynamo.guards.TensorGuards(
                *tensors, dynamic_dims_sizes=[list(t.shape) for t in tensors],
                dynamic_dims_strides=[list(t.stride()) for t in tensors])
        except (AttributeError, TypeError):         # not in this torch, or not for these tensors
            self._guards = None

    def again(self, tensors) -> bool:
        try:
            return self._guards is not None and self._guards.check(*tensors)
        except TypeError:                           # another number of them
            return False


class AdamWPlan:
    """Parameters and their optimizer state, checked once: what adamw_step updates in place.

    params, master, exp_avg, exp_avg_sq, avg_scale, sq_scale are lists of tensors (None for a
    kind that is not there); a checkpoint saves and restores their contents.  With 8-bit states
    exp_avg holds E4M3 codes of m / avg_scale and exp_avg_sq those of sqrt(v) / sq_scale, one
    scale per 128 elements.  The tensors are looked at again at each step, so `p.data = ...` is
    noticed, and refused where the number, the sizes, the types or the device are no longer the plan's,
    a tensor is not contiguous or two share memory."""

    KINDS = ("params", "exp_avg", "exp_avg_sq", "master", "avg_scale", "sq_scale")

    def __init__(self, params, exp_avg, exp_avg_sq, master, avg_scale, sq_scale):
        self.params, self.exp_avg, self.exp_avg_sq = params, exp_avg, exp_avg_sq
        self.master, self.avg_scale, self.sq_scale = master, avg_scale, sq_scale
        self.device = params[0].device
        self.numels = [p.numel() for p in params]
        self.ptype = _type(params[0], "parameters")
        self.dtype = params[0].dtype
        state = exp_avg[0].dtype
        if state not in (torch.float32, torch.float8_e4m3fn):
            raise TypeError("states must be float32 or float8_e4m3fn, got %s" % state)
        self.state = STATES["f32" if state == torch.float32 else "e4m3"]
        if (self.state == 1) != (avg_scale is not None) or (self.state == 1) != (sq_scale is not None):
            raise ValueError("avg_scale and sq_scale go with float8_e4m3fn states, and only with them")
        if master is not None and self.dtype != torch.bfloat16:
            raise ValueError("a master copy goes with bfloat16 parameters only")
        blocks = [-(-n // ADAMW_BLOCK) for n in self.numels]
        # nvfp4_adamw_tensor, an entry a row
        self._table = np.zeros((len(params), 8), np.int64)
        self._table[:, 7] = self.numels
        self._at = {}                   # the addresses in it
        self._seen, self._seen_grads, self._seen_out = _Seen(), _Seen(), _Seen()
        self._columns = [(k, kind, sizes, dtype) for k, kind, sizes, dtype in (
            (0, "params", self.numels, self.dtype), (2, "exp_avg", self.numels, state),
            (3, "exp_avg_sq", self.numels, state), (4, "master", self.numels, torch.float32),
            (5, "avg_scale", blocks, torch.float32), (6, "sq_scale", blocks, torch.float32))
            if getattr(self, kind) is not None]
        self._fill()

    def _look(self, kind, t, numel, dtype):
        if t.dtype != dtype:
            raise TypeError("%s must be %s, got %s" % (kind, dtype, t.dtype))
        if not t.is_cuda or t.device != self.device:
            raise ValueError("%s must be GPU tensors, all on one device" % kind)
        if t.numel() != numel or not t.is_contiguous():
            raise ValueError("%s must be contiguous, with %d elements, got %s"
                             % (kind, numel, tuple(t.shape)))

    def _fill(self):
        lists = [getattr(self, kind) for _, kind, _, _ in self._columns]
        flat = list(chain.from_iterable(lists))
        if set(map(len, lists)) != {len(self.numels)} or not self._seen.again(flat):
            for (_, kind, sizes, dtype), tensors in zip(self._columns, lists):
                if len(tensors) != len(sizes):
                    raise ValueError("%s: %d tensors for %d parameters" % (kind, len(tensors), len(sizes)))
                for t, n in zip(tensors, sizes):
                    self._look(kind, t, n, dtype)
            self._seen.keep(flat)
        moved = {}
        for (k, _, _, _), tensors in zip(self._columns, lists):
            now = [t.data_ptr() for t in tensors]
            if now != self._at.get(k):
                moved[k] = now
        if moved:
            self._look_apart({**self._at, **moved})
            for k, now in moved.items():
                self._table[:, k] = self._at[k] = now

    def _look_apart(self, at):
        """That no two of the tensors at these addresses share memory: a launch writes all of them."""
        parts = sorted((a, a + n * dtype.itemsize, kind) for k, kind, sizes, dtype in self._columns
                       for a, n in zip(at[k], sizes) if n)
        for (_, end, one), (start, _, other) in zip(parts, parts[1:]):
            if start < end:
                raise ValueError("%s and %s share memory" % (one, other) if one != other
                                 else "two tensors of %s share memory" % one)

    def _look_grads(self, grads) -> int:
        """The gradients' type, all of them checked."""
        if not self._seen_grads.again(grads):
            for k, g in enumerate(grads):
                if g is None:
                    raise ValueError("gradient %d is None: a plan steps all of its tensors" % k)
            _type(grads[0], "gradients")
            for g, n in zip(grads, self.numels):
                self._look("grads", g, n, grads[0].dtype)
            self._seen_grads.keep(grads)
        return TYPES[grads[0].dtype]

    def table(self, grads) -> np.ndarray:
        """The entries of nvfp4_adamw_tensor for these gradients."""
        self._fill()
        self._table[:, 1] = [g.data_ptr() for g in grads]
        return self._table


def adamw_plan(params, exp_avg=None, exp_avg_sq=None, *, master=None, avg_scale=None,
               sq_scale=None, state: str = "f32") -> AdamWPlan:
    """An AdamWPlan over `params` (float32, or bfloat16).

    Without exp_avg and exp_avg_sq the state is made here, zero: float32, or with
    state="e4m3" 8 bits plus scales.  master: a list of float32 tensors that bfloat16
    parameters are copies of, True to make them from the parameters, or None: bfloat16 parameters are
    then updated by stochastic rounding."""
    params = list(params)
    if not params:
        raise ValueError("no parameters")
    if not all(p.is_cuda for p in params):
        raise ValueError("params must be GPU tensors")
    if (exp_avg is None) != (exp_avg_sq is None):
        raise ValueError("exp_avg and exp_avg_sq come together")
    if exp_avg is None:
        if state not in STATES:
            raise ValueError("state must be one of %s" % ", ".join(STATES))
        if avg_scale is not None or sq_scale is not None:
            raise ValueError("avg_scale and sq_scale come with exp_avg and exp_avg_sq")
        dtype = torch.float32 if state == "f32" else torch.float8_e4m3fn
        zeros = lambda: [torch.zeros(p.shape, dtype=dtype, device=p.device) for p in params]
        exp_avg, exp_avg_sq = zeros(), zeros()
        if state == "e4m3":
            scales = lambda: [torch.zeros(-(-p.numel() // ADAMW_BLOCK), dtype=torch.float32,
                                          device=p.device) for p in params]
            avg_scale, sq_scale = scales(), scales()
    if master is True:
        master = [p.detach().to(torch.float32, copy=True) for p in params]
    listed = lambda v: None if v is None else list(v)
    return AdamWPlan(params, list(exp_avg), list(exp_avg_sq), listed(master), listed(avg_scale),
                     listed(sq_scale))


def adamw_step(plan: AdamWPlan, grads, *, step: int, lr: float, betas=(0.9, 0.999),
               eps: float = 1e-8, weight_decay: float = 0.01, grad_scale: torch.Tensor = None,
               amax: torch.Tensor = None, seed: int = 0) -> None:
    """One AdamW step on the plan's tensors, in place.

    grads: one tensor per parameter (None is refused: a plan steps all of its tensors), all bfloat16
    or all float32.  step: 1 for the first.
    grad_scale: float32 [1] on the GPU that multiplies the gradients (a clipping coefficient).
    amax: float32 [tensors], receives max |param| as written, for the *_from_amax calls.
    seed: of the stochastic rounding of 8-bit states and of bfloat16 parameters without a master
    copy."""
    grads = list(grads)
    if len(grads) != len(plan.params):
        raise ValueError("%d gradients for %d parameters" % (len(grads), len(plan.params)))
    kind = plan._look_grads(grads)
    like = plan.params[0]
    if grad_scale is not None:
        _vector(grad_scale, (1,), _F32, like, "grad_scale")
    if amax is not None:
        _vector(amax, (len(grads),), _F32, like, "amax")
    if not 0 <= seed < 1 << 32:
        raise ValueError("seed must be in 0 .. 2^32 - 1")
    args = AdamWArgs(lr, betas[0], betas[1], eps, weight_decay, step, seed)
    _call("nvfp4_adamw_step", like, plan.table(grads).ctypes.data, len(grads), plan.ptype, kind,
          plan.state, ctypes.byref(args), _ptr(grad_scale), _ptr(amax))
