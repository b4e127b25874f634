"""Argument checks of the training operators (no GPU): every refusal comes back as a status, or
as a Python exception, before anything reaches a device."""
from __future__ import annotations

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import nvfp4_block_scaled_amax_amd as nv
from nvfp4_block_scaled_amax_amd import train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
HEADER = os.path.join(ROOT, "include", "nvfp4_train.h")
OK, ENULL, ESHAPE, EBLOCK, EENUM, EALIGN, EHIP, EALIAS, ESCRATCH, EVALUE = range(10)
BF16, F32 = 0, 1

# fake, never dereferenced addresses, 16 MiB apart
A, B, C, D, E, F, G, H = (0x10000000 + 0x1000000 * i for i in range(8))


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_block_scaled_amax_amd import build
        build.build_library()
    return nv.lib()


def test_library_exports_what_the_header_declares(L):
    text = open(HEADER).read()
    names = set(re.findall(r"^(?:nvfp4_status|int|int64_t|const char\*)\s+(nvfp4_\w+)\s*\(", text, re.M))
    assert names == {"nvfp4_train_abi_version", "nvfp4_train_status_str", "nvfp4_layernorm_forward",
                     "nvfp4_layernorm_backward_workspace", "nvfp4_layernorm_backward",
                     "nvfp4_distill_loss_workspace", "nvfp4_distill_loss", "nvfp4_adamw_step"}
    for n in names:
        assert hasattr(L, n), n
    assert L.nvfp4_train_abi_version() == 1
    for st in (OK, ENULL, ESHAPE, EENUM, EALIGN, EHIP, EALIAS, EVALUE):
        assert L.nvfp4_train_status_str(st) != b"unknown status"
    assert L.nvfp4_train_status_str(99) == b"unknown status"


def fwd(L, x=A, xs=64, res=None, rs=64, w=B, b=C, rows=4, cols=64, t=BF16, wt=BF16, center=1,
        eps=1e-5, y=D, h=None, mean=E, rstd=F, amax=None):
    return L.nvfp4_layernorm_forward(x, xs, res, rs, w, b, rows, cols, t, wt, center, eps, y, h,
                                     mean, rstd, amax, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), ENULL), (dict(w=None), ENULL), (dict(y=None), ENULL), (dict(rstd=None), ENULL),
    (dict(mean=None), ENULL), (dict(res=G), ENULL), (dict(h=G), ENULL),
    (dict(cols=0, xs=1), ESHAPE), (dict(rows=-1), ESHAPE), (dict(xs=63), ESHAPE),
    (dict(res=G, h=H, rs=60), ESHAPE), (dict(rows=1 << 58), ESHAPE), (dict(xs=1 << 41), ESHAPE),
    (dict(cols=(1 << 30) + 1, xs=1 << 31), ESHAPE),
    (dict(t=2), EENUM), (dict(wt=-1), EENUM), (dict(eps=-1.0), EVALUE),
    (dict(eps=float("nan")), EVALUE), (dict(eps=float("inf")), EVALUE),
    (dict(x=A + 1), EALIGN), (dict(t=F32, y=D + 2), EALIGN), (dict(wt=F32, b=C + 2), EALIGN),
    (dict(rstd=F + 2), EALIGN), (dict(amax=G + 1), EALIGN),
    (dict(y=A + 2), EALIAS), (dict(y=A, xs=65), EALIAS), (dict(y=A, res=G, h=H), EALIAS),
    (dict(y=G, res=G, h=H), EALIAS), (dict(res=G, h=H, y=H), EALIAS), (dict(rstd=E + 4), EALIAS),
    (dict(mean=B), EALIAS), (dict(amax=F), EALIAS), (dict(res=G, rs=70, h=G), EALIAS)])
def test_layer_norm_forward_refuses(L, kw, status):
    assert fwd(L, **kw) == status


def bwd(L, dy=A, h=B, w=C, mean=D, rstd=E, dres=None, rows=4, cols=64, t=BF16, wt=BF16, dx=F,
        dw=G, db=G + 4096, ws=H):
    return L.nvfp4_layernorm_backward(dy, h, w, mean, rstd, dres, rows, cols, t, wt, dx, dw, db, ws,
                                      None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), ENULL), (dict(h=None), ENULL), (dict(w=None), ENULL), (dict(rstd=None), ENULL),
    (dict(dx=None), ENULL), (dict(dw=None), ENULL), (dict(ws=None), ENULL),
    (dict(cols=0), ESHAPE), (dict(rows=-2), ESHAPE), (dict(t=7), EENUM), (dict(wt=2), EENUM),
    (dict(dy=A + 1), EALIGN), (dict(ws=H + 8), EALIGN), (dict(mean=D + 2), EALIGN),
    (dict(dx=A + 2), EALIAS), (dict(dx=B), EALIAS), (dict(dw=C), EALIAS), (dict(db=G + 64), EALIAS),
    (dict(ws=F), EALIAS), (dict(dw=E), EALIAS), (dict(dres=F + 16), EALIAS)])
def test_layer_norm_backward_refuses(L, kw, status):
    assert bwd(L, **kw) == status


def test_workspace_sizes_need_no_gpu(L):
    assert L.nvfp4_layernorm_backward_workspace(0, 64) == 0
    assert L.nvfp4_layernorm_backward_workspace(-1, 64) == 0
    assert L.nvfp4_layernorm_backward_workspace(5, 0) == 0
    assert L.nvfp4_layernorm_backward_workspace(1, 64) >= 2 * 64 * 4
    assert L.nvfp4_distill_loss_workspace(0, 1000) == 0
    assert L.nvfp4_distill_loss_workspace(1, 128000) > 0


def kl(L, s=A, ss=100, t=B, ts=100, w=C, rows=2, vocab=100, st=BF16, tt=BF16, temp=1.0, loss=D,
       grad=E, gs=100, ws=F):
    return L.nvfp4_distill_loss(s, ss, t, ts, w, rows, vocab, st, tt, temp, loss, grad, gs, ws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(s=None), ENULL), (dict(t=None), ENULL), (dict(loss=None), ENULL),
    (dict(vocab=100000, ss=100000, ts=100000, gs=100000, ws=None), ENULL),
    (dict(vocab=0), ESHAPE), (dict(rows=-1), ESHAPE), (dict(ss=99), ESHAPE), (dict(ts=99), ESHAPE),
    (dict(gs=99), ESHAPE), (dict(st=2), EENUM), (dict(tt=-1), EENUM),
    (dict(temp=0.0), EVALUE), (dict(temp=-1.0), EVALUE), (dict(temp=float("nan")), EVALUE),
    (dict(temp=float("inf")), EVALUE), (dict(temp=1e-39), EVALUE),
    (dict(s=A + 1), EALIGN), (dict(tt=F32, t=B + 2), EALIGN), (dict(loss=D + 2), EALIGN),
    (dict(vocab=100000, ss=100000, ts=100000, gs=100000, ws=F + 4), EALIGN),
    (dict(grad=A + 2), EALIAS), (dict(grad=A, gs=101), EALIAS), (dict(grad=B), EALIAS),
    (dict(loss=C), EALIAS), (dict(loss=E + 8), EALIAS),
    (dict(vocab=100000, ss=100000, ts=100000, gs=100000, ws=E), EALIAS)])
def test_distill_loss_refuses(L, kw, status):
    assert kl(L, **kw) == status


def adamw(L, n=100, ptype=F32, gtype=F32, state=0, count=1, second=None, args=None, scale=None,
          amax=None, tensors=True, **field):
    first = dict(param=A, grad=B, exp_avg=C, exp_avg_sq=D, numel=n)
    first.update(field)
    rows = [first] + ([second] if second else [])
    table = (train.AdamWTensor * len(rows))(*[train.AdamWTensor(**r) for r in rows])
    a = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1, seed=0)
    a.update(args or {})
    return L.nvfp4_adamw_step(table if tensors else None, max(count, len(rows)) if count > 0 else count,
                              ptype, gtype, state, ctypes.byref(train.AdamWArgs(**a)), scale, amax,
                              None)


@pytest.mark.parametrize("kw,status", [
    (dict(param=None), ENULL), (dict(grad=None), ENULL), (dict(exp_avg=None), ENULL),
    (dict(exp_avg_sq=None), ENULL), (dict(state=1), ENULL), (dict(state=1, avg_scale=E), ENULL),
    (dict(tensors=False), ENULL),
    (dict(ptype=BF16, master=E, second=dict(param=F, grad=G, exp_avg=H, exp_avg_sq=H + 4096, numel=4)),
     ENULL),
    (dict(n=-1), ESHAPE), (dict(n=(1 << 36) + 1), ESHAPE), (dict(count=-1), ESHAPE),
    (dict(ptype=2), EENUM), (dict(gtype=-1), EENUM), (dict(state=2), EENUM), (dict(master=E), EENUM),
    (dict(args=dict(beta1=1.0)), EVALUE), (dict(args=dict(beta2=-0.1)), EVALUE),
    (dict(args=dict(eps=-1e-8)), EVALUE), (dict(args=dict(step=0)), EVALUE),
    (dict(args=dict(step=1 << 32)), EVALUE), (dict(args=dict(lr=float("nan"))), EVALUE),
    (dict(args=dict(weight_decay=float("inf"))), EVALUE),
    (dict(param=A + 2), EALIGN), (dict(ptype=BF16, param=A + 1), EALIGN), (dict(exp_avg=C + 2), EALIGN),
    (dict(scale=E + 2), EALIGN), (dict(amax=E + 1), EALIGN),
    (dict(exp_avg=D + 4), EALIAS), (dict(grad=A), EALIAS), (dict(amax=C), EALIAS),
    (dict(scale=A + 8), EALIAS), (dict(state=1, avg_scale=E, sq_scale=E), EALIAS)])
def test_adamw_refuses(L, kw, status):
    assert adamw(L, **kw) == status


def test_nothing_to_do_is_not_an_error(L):
    """No row or no tensor: nothing is enqueued, so these succeed without a GPU."""
    assert fwd(L, x=None, y=None, mean=None, rstd=None, rows=0) == OK
    assert kl(L, s=None, t=None, loss=None, rows=0) == OK
    assert adamw(L, count=0) == OK
    assert adamw(L, n=0, param=None, grad=None, exp_avg=None, exp_avg_sq=None) == OK


def test_python_refusals():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    w = torch.ones(32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        nv.layer_norm(x, w)
    with pytest.raises(ValueError, match="GPU"):
        nv.layer_norm_backward(x, x, w, torch.zeros(4), torch.ones(4))
    with pytest.raises(ValueError, match="GPU"):
        nv.distill_loss(x, x)
    with pytest.raises(ValueError, match="GPU"):
        nv.adamw_plan([x])
    with pytest.raises(ValueError, match="no parameters"):
        nv.adamw_plan([])


PROGRAM = r"""
#include <stdio.h>
#include <string.h>
#include "nvfp4_train.h"
#define CHECK(cond) do { if (!(cond)) { printf("FAIL %s\n", #cond); return 1; } } while (0)
int main(void) {
  float* f = (float*)(uintptr_t)0x100000;
  uint16_t* x = (uint16_t*)(uintptr_t)0x900000;
  nvfp4_adamw_tensor t = {0};
  nvfp4_adamw_args a = {1e-3, 0.9, 0.999, 1e-8, 0.0, 0, 0};
  CHECK(nvfp4_train_abi_version() == NVFP4_TRAIN_ABI_VERSION);
  CHECK(strcmp(nvfp4_train_status_str(NVFP4_ERR_VALUE), "unknown status") != 0);
  CHECK(nvfp4_layernorm_forward(NULL, 8, NULL, 8, x, NULL, 1, 8, NVFP4_T_BF16, NVFP4_T_BF16, 0,
                                1e-5f, x, NULL, NULL, f, NULL, NULL) == NVFP4_ERR_NULL);
  CHECK(nvfp4_layernorm_backward(x, x, x, f, f, NULL, 1, 0, NVFP4_T_BF16, NVFP4_T_BF16, x, x, x, f,
                                 NULL) == NVFP4_ERR_SHAPE);
  CHECK(nvfp4_distill_loss(x, 8, x, 8, NULL, 1, 8, NVFP4_T_BF16, NVFP4_T_BF16, 0.0f, f, NULL, 8,
                           NULL, NULL) == NVFP4_ERR_VALUE);
  CHECK(nvfp4_adamw_step(&t, 1, NVFP4_T_F32, NVFP4_T_F32, NVFP4_STATE_F32, &a, NULL, NULL, NULL)
        == NVFP4_ERR_VALUE);
  printf("c consumer ok\n");
  return 0;
}
"""


def test_c_program_compiles_links_and_runs(tmp_path, L):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    src, exe = tmp_path / "consumer.c", tmp_path / "consumer"
    src.write_text(PROGRAM)
    libdir = os.path.dirname(nv.LIB_PATH)
    cmd = [gcc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROCM, "include"), str(src), "-o", str(exe), "-L", libdir,
           "-lnvfp4_amax", "-Wl,-rpath," + libdir, "-L", os.path.join(ROCM, "lib"),
           "-Wl,-rpath," + os.path.join(ROCM, "lib"), "-lamdhip64"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "c consumer ok" in r.stdout


def test_a_library_of_one_source_links():
    """flags() compile and link a shared library by themselves (tests/hw is built with them)."""
    import tempfile
    from nvfp4_block_scaled_amax_amd import build
    with tempfile.TemporaryDirectory() as work:
        src, lib = os.path.join(work, "one.hip"), os.path.join(work, "one.so")
        with open(src, "w") as f:
            f.write('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
        subprocess.run([build.hipcc()] + build.flags() + ["-o", lib, src], check=True, capture_output=True)
        assert ctypes.CDLL(lib).one() == 1


class OnTheGpu:
    """What an AdamWPlan looks at of a GPU tensor."""

    def __init__(self, numel, dtype=torch.float32, at=A, contiguous=True, device=0):
        self.dtype, self.shape, self.is_cuda = dtype, (numel,), device >= 0
        self.device = torch.device("cuda", device) if device >= 0 else torch.device("cpu")
        self._numel, self._at, self._contiguous = numel, at, contiguous

    def numel(self):
        return self._numel

    def data_ptr(self):
        return self._at

    def is_contiguous(self):
        return self._contiguous

    def get_device(self):
        return self.device.index if self.is_cuda else -1


PLAN = {"params": (torch.bfloat16, 1600), "exp_avg": (torch.float8_e4m3fn, 1600),
        "exp_avg_sq": (torch.float8_e4m3fn, 1600), "master": (torch.float32, 1600),
        "avg_scale": (torch.float32, 13), "sq_scale": (torch.float32, 13)}


@pytest.mark.parametrize("change,error", [
    (dict(numel=12), ValueError), (dict(numel=3000), ValueError), (dict(dtype=torch.float16), TypeError),
    (dict(contiguous=False), ValueError), (dict(device=1), ValueError), (dict(device=-1), ValueError)])
@pytest.mark.parametrize("kind", list(PLAN))
def test_a_plan_refuses_tensors_that_changed_where_they_are(kind, change, error):
    """A tensor of another size, type, order or device at the address that the plan knows (a view of
    it; memory that was freed and taken again) is refused at the next step, before anything is
    enqueued; one that is the same but for its address is taken."""
    lists = {k: [OnTheGpu(n, dtype, B + 0x100000 * i + 0x10000 * j) for j in range(3)]
             for i, (k, (dtype, n)) in enumerate(PLAN.items())}
    plan = train.AdamWPlan(**lists)
    grads = [OnTheGpu(1600, torch.bfloat16, G + 0x10000 * j) for j in range(3)]
    table = plan.table(grads).copy()
    assert (table == plan.table(grads)).all()
    dtype, n = PLAN[kind]
    held = lists[kind][1]
    lists[kind][1] = OnTheGpu(**{**dict(numel=n, dtype=dtype, at=held.data_ptr()), **change})
    for _ in range(2):
        with pytest.raises(error, match=kind):
            plan.table(grads)
    lists[kind][1] = OnTheGpu(n, dtype, H)
    again = plan.table(grads)
    assert (again != table).sum() == 1 and (again[1] == H).sum() == 1
    lists[kind][1] = held
    assert (plan.table(grads) == table).all()


def test_tensors_are_recognized_by_more_than_their_addresses():
    """What was checked once is recognized, also elsewhere in memory; a view of it at the same address
    with another size, order or type is not, nor is another number of tensors."""
    seen = train._Seen()
    ts = [torch.zeros(40, 40), torch.nn.Parameter(torch.zeros(300)), torch.zeros(7, dtype=torch.bfloat16)]
    assert not seen.again(ts)
    seen.keep(ts)
    assert seen.again(ts)
    whole = ts[0].data
    ts[0].data = whole.clone()
    assert seen.again(ts)
    for other in (whole.t(), whole[:2], whole.view(torch.int32), whole.view(torch.bfloat16)[:, :40],
                  whole.as_strided((40, 40), (1, 1)), whole.to("meta")):
        assert not seen.again([other] + ts[1:])
    ts[0].data = whole.t()                    # the same object
    assert not seen.again(ts)
    ts[0].data = whole
    assert not seen.again(ts[:2]) and not seen.again(ts + ts[:1]) and not seen.again(ts[:2] + [None])
    with torch.no_grad():
        assert seen.again(ts)
    seen.keep([object()])                     # nothing that can be compared: never recognized
    assert not seen.again([object()])


def test_a_missing_gradient_is_named():
    """None in the list of gradients (a parameter that the step did not use) is refused by its place."""
    plan = train.AdamWPlan([OnTheGpu(8, at=A), OnTheGpu(8, at=B)], [OnTheGpu(8, at=C), OnTheGpu(8, at=D)],
                           [OnTheGpu(8, at=E), OnTheGpu(8, at=F)], None, None, None)
    g = OnTheGpu(8, at=G)
    for grads, place in (([None, g], 0), ([g, None], 1)):
        with pytest.raises(ValueError, match="gradient %d is None" % place):
            train.adamw_step(plan, grads, step=1, lr=0.1)


def test_a_plan_refuses_tensors_that_share_memory():
    """A parameter listed twice (tied weights), a state that is another's, parts that overlap: the
    workgroups of one launch would race for them.  Neighbours in one buffer and empty tensors do not."""
    def plan(params, avg, sq):
        return train.AdamWPlan(params, avg, sq, None, None, None).table(grads)
    grads = [OnTheGpu(100, at=G), OnTheGpu(100, at=H)]
    apart = lambda at: [OnTheGpu(100, at=at), OnTheGpu(100, at=at + 400)]
    plan(apart(A), apart(B), apart(C))
    for params, avg, sq in ((apart(A)[:1] * 2, apart(B), apart(C)), (apart(A), apart(B)[:1] * 2, apart(C)),
                            (apart(A), apart(B), apart(B)), (apart(A), apart(A + 796), apart(C)),
                            ([OnTheGpu(100, at=A), OnTheGpu(100, at=A + 396)], apart(B), apart(C))):
        with pytest.raises(ValueError, match="share memory"):
            plan(params, avg, sq)
    later = train.AdamWPlan(apart(A), apart(B), apart(C), None, None, None)
    later.exp_avg[1] = later.exp_avg[0]
    for _ in range(2):
        with pytest.raises(ValueError, match="share memory"):
            later.table(grads)
    none = [OnTheGpu(0, at=0), OnTheGpu(0, at=0)]
    train.AdamWPlan(none, none, none, None, None, None)
