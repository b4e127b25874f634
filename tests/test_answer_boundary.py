"""Argument checks of the operators of a step on a model's own answers (no GPU): every refusal comes back
as a status, or as a Python exception, before anything reaches a device."""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amax_amd as nv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
HEADER = os.path.join(ROOT, "include", "nvfp4_answer.h")
OK, ENULL, ESHAPE, EBLOCK, EENUM, EALIGN, EHIP, EALIAS, ESCRATCH, EVALUE = range(10)
BF16, F32 = 0, 1
I32, I64 = 0, 1

# fake, never dereferenced addresses, 16 MiB apart
A, B, C, D, E, F, G, H, J = (0x10000000 + 0x1000000 * i for i in range(9))


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_block_scaled_amax_amd import build
        build.build_library()
    return nv.lib()


def test_library_exports_what_the_header_declares(L):
    text = open(HEADER).read()
    names = set(re.findall(r"^(?:nvfp4_status|int|int64_t|const char\*)\s+(nvfp4_\w+)\s*\(", text, re.M))
    assert names == {"nvfp4_answer_abi_version", "nvfp4_packed_matvec",
                     "nvfp4_token_logprobs_workspace", "nvfp4_token_logprobs",
                     "nvfp4_token_logprobs_backward", "nvfp4_grad_norm", "nvfp4_clip_grads"}
    for n in names:
        assert hasattr(L, n), n
    assert L.nvfp4_answer_abi_version() == 1
    for name, value in (("MATVEC_MAX_ROWS", nv.MATVEC_MAX_ROWS), ("LOGPROBS_MAX", nv.LOGPROBS_MAX)):
        assert int(re.search(r"#define NVFP4_%s (\d+)" % name, text).group(1)) == value


def matvec(L, x=A, xs=64, codes=B, scales=C, alpha=D, expert=None, tokens=4, picks=1, experts=1, rows=32,
           cols=64, xt=BF16, yt=BF16, it=I32, y=F):
    return L.nvfp4_packed_matvec(x, xs, codes, scales, alpha, expert, tokens, picks, experts, rows, cols,
                                 xt, yt, it, y, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), ENULL), (dict(codes=None), ENULL), (dict(scales=None), ENULL), (dict(alpha=None), ENULL),
    (dict(y=None), ENULL),
    (dict(tokens=-1), ESHAPE), (dict(tokens=1025), ESHAPE), (dict(rows=0), ESHAPE), (dict(cols=0, xs=1), ESHAPE),
    (dict(cols=40), ESHAPE), (dict(xs=63), ESHAPE), (dict(picks=2), ESHAPE), (dict(experts=2), ESHAPE),
    (dict(expert=E, picks=0), ESHAPE), (dict(expert=E, picks=257), ESHAPE),
    (dict(expert=E, experts=65536), ESHAPE), (dict(expert=E, experts=0), ESHAPE),
    (dict(expert=E, experts=65535, rows=1 << 26, cols=1 << 27, xs=1 << 27), ESHAPE),
    (dict(rows=(1 << 26) + 1), ESHAPE), (dict(xs=1 << 41), ESHAPE), (dict(cols=(1 << 27) + 16, xs=1 << 28), ESHAPE),
    (dict(xt=2), EENUM), (dict(yt=-1), EENUM), (dict(it=2), EENUM),
    (dict(x=A + 1), EALIGN), (dict(xt=F32, x=A + 2), EALIGN), (dict(codes=B + 4), EALIGN),
    (dict(alpha=D + 2), EALIGN), (dict(yt=F32, y=F + 2), EALIGN),
    (dict(expert=E + 4, it=I64), EALIGN), (dict(expert=E + 2), EALIGN),
    (dict(y=A + 128), EALIAS), (dict(y=B), EALIAS), (dict(y=C), EALIAS), (dict(y=D), EALIAS),
    (dict(expert=E, y=E), EALIAS)])
def test_packed_matvec_refuses(L, kw, status):
    assert matvec(L, **kw) == status


def logprobs(L, x=A, xs=100, t=B, rows=2, vocab=100, given=1, top=2, ty=BF16, it=I64, temp=1.0, logp=C, ent=D,
             tl=E, ti=F, st=G, ws=H):
    return L.nvfp4_token_logprobs(x, xs, t, rows, vocab, given, top, ty, it, temp, logp, ent, tl, ti, st, ws, None)


LONG = dict(vocab=100000, xs=100000)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), ENULL), (dict(t=None), ENULL), (dict(logp=None), ENULL), (dict(tl=None), ENULL),
    (dict(ti=None), ENULL), (dict(st=None), ENULL), (dict(ws=None, **LONG), ENULL),
    (dict(vocab=0), ESHAPE), (dict(vocab=(1 << 28) + 1, xs=1 << 29), ESHAPE), (dict(rows=-1), ESHAPE),
    (dict(xs=99), ESHAPE), (dict(given=-1), ESHAPE), (dict(given=65), ESHAPE), (dict(top=-1), ESHAPE),
    (dict(top=65), ESHAPE), (dict(vocab=1, top=2), ESHAPE), (dict(rows=(1 << 30) + 1), ESHAPE),
    (dict(ty=2), EENUM), (dict(it=-1), EENUM), (dict(temp=0.0), EVALUE), (dict(temp=-2.0), EVALUE),
    (dict(temp=float("nan")), EVALUE), (dict(temp=float("inf")), EVALUE), (dict(temp=1e-39), EVALUE),
    (dict(x=A + 1), EALIGN), (dict(ty=F32, x=A + 2), EALIGN), (dict(t=B + 4), EALIGN), (dict(it=I32, t=B + 2), EALIGN),
    (dict(logp=C + 2), EALIGN), (dict(ent=D + 1), EALIGN), (dict(tl=E + 2), EALIGN), (dict(ti=F + 4), EALIGN),
    (dict(st=G + 2), EALIGN), (dict(ws=H + 8, **LONG), EALIGN),
    (dict(logp=A), EALIAS), (dict(ent=B + 8), EALIAS), (dict(tl=C + 4), EALIAS), (dict(ti=E), EALIAS),
    (dict(st=F + 16), EALIAS), (dict(ws=G, **LONG), EALIAS)])
def test_token_logprobs_refuses(L, kw, status):
    assert logprobs(L, **kw) == status


LONG_ROWS = r"""
import ctypes, sys
import nvfp4_block_scaled_amax_amd as nv
L, n = nv.lib(), ctypes.c_int(0)
if ctypes.CDLL("libamdhip64.so").hipGetDeviceCount(ctypes.byref(n)) == 0 and n.value:
    sys.exit(77)                                    # nothing may be launched on these addresses
at = [0x10000000000 * i for i in range(1, 8)]
for rows, vocab in ((512, 328320), (513, 328319), (513, 328320), (600, 400000), (1024, 1 << 20), (1 << 14, 1 << 24)):
    for top in (0, 64):
        print(rows, vocab, top, L.nvfp4_token_logprobs_workspace(rows, vocab, top),
              L.nvfp4_token_logprobs(at[0], vocab, None, rows, vocab, 0, top, 0, 1, 1.0, None, at[2], at[3], at[4],
                                     at[5], None, None), flush=True)
"""


def test_token_logprobs_of_many_long_rows_return(L):
    """More rows than are shared among workgroups, however long: no workspace, and the call comes back (without a
    device, with the status of a launch that failed)."""
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", LONG_ROWS], env=env, capture_output=True, text=True, timeout=120)
    if r.returncode == 77:
        pytest.skip("a GPU is there all the same")
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr)
    lines = r.stdout.split("\n")[:-1]
    assert len(lines) == 12 and all(line.split()[3:] == ["0", str(EHIP)] for line in lines), r.stdout
    assert L.nvfp4_token_logprobs_workspace(2 ** 63 - 1, 2 ** 63 - 1, 64) == 0


def back(L, x=A, xs=100, t=B, st=C, ent=D, dl=E, dh=F, rows=2, vocab=100, given=1, ty=BF16, it=I64, temp=1.0, g=G,
         gs=100):
    return L.nvfp4_token_logprobs_backward(x, xs, t, st, ent, dl, dh, rows, vocab, given, ty, it, temp, g, gs, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), ENULL), (dict(t=None), ENULL), (dict(st=None), ENULL), (dict(dl=None), ENULL),
    (dict(g=None), ENULL), (dict(ent=None), ENULL),
    (dict(vocab=0), ESHAPE), (dict(rows=-1), ESHAPE), (dict(xs=99), ESHAPE), (dict(gs=99), ESHAPE),
    (dict(given=0), ESHAPE), (dict(given=65), ESHAPE), (dict(rows=(1 << 30) + 1), ESHAPE),
    (dict(ty=3), EENUM), (dict(it=2), EENUM), (dict(temp=0.0), EVALUE), (dict(temp=float("inf")), EVALUE),
    (dict(x=A + 1), EALIGN), (dict(g=G + 1), EALIGN), (dict(t=B + 4), EALIGN), (dict(dl=E + 2), EALIGN),
    (dict(st=C + 2), EALIGN), (dict(ent=D + 2), EALIGN), (dict(dh=F + 2), EALIGN),
    (dict(g=A + 2), EALIAS), (dict(g=A, gs=101), EALIAS), (dict(g=B), EALIAS), (dict(g=C), EALIAS),
    (dict(g=D), EALIAS), (dict(g=E), EALIAS), (dict(g=F), EALIAS)])
def test_token_logprobs_backward_refuses(L, kw, status):
    assert back(L, **kw) == status


def table(*entries):
    return np.array(entries, np.int64).reshape(-1, 2)


def norm(L, entries=((A, 100),), count=None, ty=F32, most=1.0, eps=1e-6, to=B, scale=C, ws=D):
    t = table(*entries)
    return L.nvfp4_grad_norm(t.ctypes.data if len(t) else None, len(t) if count is None else count, ty, most, eps, to,
                             scale, ws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(entries=((0, 100),)), ENULL), (dict(entries=(), count=1), ENULL), (dict(to=None), ENULL), (dict(ws=None), ENULL),
    (dict(count=-1), ESHAPE), (dict(count=(1 << 24) + 1), ESHAPE), (dict(entries=((A, -1),)), ESHAPE),
    (dict(entries=((A, (1 << 36) + 1),)), ESHAPE), (dict(ty=2), EENUM), (dict(most=-1.0), EVALUE),
    (dict(most=float("nan")), EVALUE), (dict(most=float("inf")), EVALUE), (dict(eps=-1e-9), EVALUE),
    (dict(entries=((A + 2, 4),)), EALIGN), (dict(ty=BF16, entries=((A + 1, 4),)), EALIGN), (dict(to=B + 2), EALIGN),
    (dict(scale=C + 1), EALIGN), (dict(ws=D + 8), EALIGN),
    (dict(to=A + 8), EALIAS), (dict(scale=B), EALIAS), (dict(ws=A), EALIAS), (dict(scale=D + 16), EALIAS)])
def test_grad_norm_refuses(L, kw, status):
    assert norm(L, **kw) == status


def clip(L, entries=((A, 100), (B, 50)), out=None, ty=F32, scale=E):
    t = table(*entries)
    o = None if out is None else table(*out)
    return L.nvfp4_clip_grads(t.ctypes.data, None if o is None else o.ctypes.data, len(t), ty, scale, None)


@pytest.mark.parametrize("kw,status", [
    (dict(entries=((0, 100),)), ENULL), (dict(scale=None), ENULL), (dict(out=((C, 100), (0, 50))), ENULL),
    (dict(entries=((A, -1),)), ESHAPE), (dict(out=((C, 100), (D, 51))), ESHAPE), (dict(ty=-1), EENUM),
    (dict(entries=((A + 1, 4),)), EALIGN), (dict(out=((C, 100), (D + 2, 50))), EALIGN), (dict(scale=E + 2), EALIGN),
    (dict(scale=A + 8), EALIAS), (dict(out=((A + 4, 100), (D, 50))), EALIAS),
    (dict(out=((C, 100), (D, 50)), scale=D + 4), EALIAS),
    (dict(entries=((A, 100), (A, 100))), EALIAS), (dict(entries=((B, 4), (A, 100), (A + 396, 2))), EALIAS),
    (dict(out=((C, 100), (C + 200, 50))), EALIAS), (dict(out=((B, 100), (A, 50))), EALIAS),
    (dict(out=((C, 100), (A, 50))), EALIAS), (dict(entries=((A, 100), (A, 100)), out=((A, 100), (C, 100))), EALIAS)])
def test_clip_grads_refuses(L, kw, status):
    assert clip(L, **kw) == status


def test_nothing_to_do_is_not_an_error(L):
    """No row or no tensor: nothing is enqueued, so these succeed without a GPU."""
    assert matvec(L, x=None, y=None, tokens=0) == OK
    assert logprobs(L, x=None, logp=None, st=None, rows=0) == OK
    assert back(L, x=None, g=None, rows=0) == OK
    assert clip(L, entries=((0, 0),)) == OK


def test_workspace_sizes_need_no_gpu(L):
    assert L.nvfp4_token_logprobs_workspace(0, 100000, 5) == 0
    assert L.nvfp4_token_logprobs_workspace(1, 0, 5) == 0
    assert L.nvfp4_token_logprobs_workspace(4096, 100000, 5) == 0
    assert L.nvfp4_token_logprobs_workspace(1, 128000, 64) > 0
    macro = re.search(r"#define NVFP4_GRAD_NORM_WORKSPACE\(count\) (.*)", open(HEADER).read()).group(1)
    for count in (0, 1, 199, 200, 201, 100000):
        assert nv.grad_norm_workspace(count) == eval(macro.replace("(int64_t)(count) /", "count //"))


def test_python_refusals():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    c, s, a = torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8), torch.zeros(1)
    with pytest.raises(ValueError, match="GPU"):
        nv.packed_matvec(x, c, s, a)
    with pytest.raises(ValueError, match="GPU"):
        nv.token_logprobs(x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="GPU"):
        nv.token_logprobs_backward(x, torch.zeros(4, dtype=torch.int64), torch.zeros(4, 2), torch.zeros(4))


PROGRAM = r"""
#include <stdio.h>
#include "nvfp4_answer.h"
#define CHECK(cond) do { if (!(cond)) { printf("FAIL %s\n", #cond); return 1; } } while (0)
int main(void) {
  float* f = (float*)(uintptr_t)0x100000;
  uint8_t* b = (uint8_t*)(uintptr_t)0x900000;
  nvfp4_grad_tensor t = {0};
  CHECK(nvfp4_answer_abi_version() == NVFP4_ANSWER_ABI_VERSION);
  CHECK(nvfp4_packed_matvec(b, 32, b, b, f, NULL, 1, 1, 1, 8, 30, NVFP4_T_BF16, NVFP4_T_BF16, NVFP4_I32, f,
                            NULL) == NVFP4_ERR_SHAPE);
  CHECK(nvfp4_token_logprobs(b, 8, NULL, 1, 8, 0, 0, NVFP4_T_BF16, NVFP4_I64, 0.0f, NULL, f, NULL, NULL, f,
                             NULL, NULL) == NVFP4_ERR_VALUE);
  CHECK(nvfp4_token_logprobs_backward(b, 8, b, f, f, f, f, 1, 8, 0, NVFP4_T_BF16, NVFP4_I64, 1.0f, b, 8, NULL)
        == NVFP4_ERR_SHAPE);
  CHECK(nvfp4_grad_norm(&t, 1, NVFP4_T_F32, -1.0, 0.0, f, NULL, f, NULL) == NVFP4_ERR_VALUE);
  CHECK(nvfp4_clip_grads(&t, NULL, 1, NVFP4_T_F32, NULL, NULL) == NVFP4_ERR_NULL);
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
