"""Layer norm forward and backward on the GPU against the formulas in 64 bits.

Tolerances.  u = 2^-24.  A sum of n terms is taken over at most s = 8 * ceil(n / 8192) + 24
sequential and tree additions per element (a lane's own terms, then the lanes' and wavefronts'
partial sums), so it is off by at most s u times the sum of magnitudes; every further operation
adds u.  A bf16 output adds half a step: half the type's eps times its value at the most.
"""
from __future__ import annotations

import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {T: torch.finfo(T).eps / 2 for T in (torch.bfloat16, torch.float32)}     # 2^-8, 2^-24
BF, F = torch.bfloat16, torch.float32


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_block_scaled_amax_amd as m
    m.lib()
    return m


def steps(n):
    return 8 * -(-n // 8192) + 24


def randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def inputs(rows, cols, T, W, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed + 1000 * rows + cols)
    x = (randn(gen, rows, cols) * torch.exp(0.5 * randn(gen, cols)) + 0.3).to(T)
    return (x, randn(gen, rows, cols).to(T), (1 + 0.3 * randn(gen, cols)).to(W),
            (0.2 * randn(gen, cols)).to(W), gen)


def near(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g times the tolerance" % (
        what, int(bad.sum()), bad.numel(), float(((got - want).abs() / tol)[bad].max()))


def forward_reference(h, w, b, eps, center):
    h = h.double()
    mean = h.mean(-1, keepdim=True) if center else torch.zeros_like(h[..., :1])
    d = h - mean
    rstd = (d.square().mean(-1, keepdim=True) + eps) ** -0.5
    y = d * rstd * w.double() + (0.0 if b is None else b.double())
    return y, mean, rstd


def check_forward(nv, x, r, w, b, center, eps=1e-5, **out):
    T, cols = x.dtype, x.shape[-1]
    amax = torch.full((1,), -1.0, device="cuda")
    y, h, mean, rstd = nv.layer_norm(x, w, b, residual=r, center=center, eps=eps, amax=amax, **out)
    want_h = x if r is None else (x.float() + r.float()).to(T)
    assert torch.equal(h, want_h)
    wy, wmean, wrstd = forward_reference(want_h, w, b, eps, center)
    s = steps(cols)
    size = want_h.double().abs().mean(-1, keepdim=True)
    off_mean = (s + 2) * U * size * center
    if center:
        near(mean[..., None], wmean, off_mean, "mean")
    # the variance is off by its own sum and, in second order, by the mean's error
    off_rstd = wrstd * ((s + 8) * U + (off_mean * wrstd) ** 2)
    near(rstd[..., None], wrstd, off_rstd, "rstd")
    scaled = (wy - (0.0 if b is None else b.double())).abs()
    tol = (HALF[T] * wy.abs() + scaled * ((s + 14) * U + (off_mean * wrstd) ** 2)
           + off_mean * wrstd * w.double().abs() + 2 * U * wy.abs()) * (1 + HALF[T]) + 1e-40
    near(y, wy, tol, "y")
    assert amax.item() == (y.float().abs().max().item() if y.numel() else 0.0)
    return y, h, mean, rstd


@pytest.mark.parametrize("T,W", [(BF, BF), (BF, F), (F, F), (F, BF)], ids=str)
@pytest.mark.parametrize("cols", [1, 2, 7, 8, 9, 64, 511, 512, 513, 1024, 1031, 2047, 2048, 2056, 4095,
                                  4096, 5120, 8191, 8192, 8200, 16383, 16384, 16385, 16392, 40001])
def test_forward(nv, cols, T, W):
    for rows in (1, 5, 67):
        say("[norm] forward", rows, cols, T, W)
        x, r, w, b, _ = inputs(rows, cols, T, W)
        check_forward(nv, x, None, w, b, True)
        check_forward(nv, x, r, w, None, False)
        check_forward(nv, x, r, w, b, True)


def test_forward_more_rows_than_workgroups(nv):
    for cols in (40, 2048, 20000):
        x, r, w, b, _ = inputs(2500 if cols > 40 else 9001, cols, BF, BF)
        check_forward(nv, x, r, w, b, True)


def backward_reference(dy, h, w, mean, rstd, dres):
    dy, h, w = dy.double(), h.double(), w.double()
    rstd = rstd.double()[..., None]
    xh = (h - (0.0 if mean is None else mean.double()[..., None])) * rstd
    g = dy * w
    c1 = 0.0 if mean is None else g.mean(-1, keepdim=True)
    c2 = (g * xh).mean(-1, keepdim=True)
    dx = rstd * (g - c1 - xh * c2) + (0.0 if dres is None else dres.double())
    return dx, (dy * xh).sum(0), dy.sum(0), g, xh, c1, c2


def check_backward(nv, dy, h, w, mean, rstd, dres, **out):
    T, cols, rows = dy.dtype, dy.shape[-1], dy.shape[0]
    want, dw, db, g, xh, c1, c2 = backward_reference(dy, h, w, mean, rstd, dres)
    dy0, h0 = dy.clone(), h.clone()
    res0 = None if dres is None else dres.double()
    dx, gw, gb = nv.layer_norm_backward(dy, h, w, mean, rstd, dres=dres, **out)
    s = steps(cols)
    size = rstd.double()[..., None] * (g.abs() + (c1 if mean is None else g.abs().mean(-1, keepdim=True))
                                       + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
    # xh itself is off by u of |h| rstd (the subtraction) and of |xh| (the product)
    lever = rstd.double()[..., None] * h0.double().abs() * U
    tol = (HALF[T] * want.abs() + (s + 12) * U * size
           + rstd.double()[..., None] * lever * (c2.abs() + g.abs().mean(-1, keepdim=True) * xh.abs())
           + 2 * U * ((0.0 if res0 is None else res0.abs()) + want.abs())) * (1 + HALF[T]) + 1e-40
    near(dx, want, tol, "dx")
    depth = rows + 64
    near(gw, dw, (HALF[w.dtype] * dw.abs() + depth * U * (dy0.double() * xh).abs().sum(0)
                  + (dy0.double().abs() * lever).sum(0)) * (1 + HALF[w.dtype]) + 1e-40, "dweight")
    if gb is not None:
        near(gb, db, (HALF[w.dtype] * db.abs() + depth * U * dy0.double().abs().sum(0))
             * (1 + HALF[w.dtype]) + 1e-40, "dbias")
    return dx, gw, gb


@pytest.mark.parametrize("T,W", [(BF, BF), (BF, F), (F, F), (F, BF)], ids=str)
@pytest.mark.parametrize("cols", [1, 7, 8, 9, 511, 512, 520, 1024, 1031, 2048, 2055, 4096, 4104, 8191, 8192,
                                  14336, 16383, 16384, 16392, 40001])
def test_backward(nv, cols, T, W):
    for rows in (1, 6, 70):
        say("[norm] backward", rows, cols, T, W)
        h, dres, w, _, gen = inputs(rows, cols, T, W)
        dy = (0.01 * randn(gen, rows, cols)).to(T)
        dres = (0.01 * dres.float()).to(T)
        for center in (True, False):
            _, mean, rstd = forward_reference(h, w, None, 1e-5, center)
            mean = mean[:, 0].float() if center else None
            rstd = rstd[:, 0].float()
            check_backward(nv, dy, h, w, mean, rstd, dres)
            dx, _, gb = check_backward(nv, dy, h, w, mean, rstd, None, bias=False)
            assert gb is None


def test_backward_more_rows_than_workgroups(nv):
    for rows, cols in ((5000, 256), (1500, 2048), (700, 8192), (600, 20000)):
        h, dres, w, _, gen = inputs(rows, cols, BF, BF)
        dy = (0.01 * randn(gen, rows, cols)).to(BF)
        _, mean, rstd = forward_reference(h, w, None, 1e-5, True)
        check_backward(nv, dy, h, w, mean[:, 0].float(), rstd[:, 0].float(), dres)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("cols", [9, 100, 3000])
def test_gradient_against_differences(nv, cols, center):
    """Directional differences of the forward formula in 64 bits, through a weighted sum of y and
    of h (the residual stream), against the kernel's gradients.  The differences' own error
    (step 1e-4: third derivatives times 1e-8) is far below the gradient's 32-bit one."""
    rows = 3
    x, _, w, b, gen = inputs(rows, cols, F, F)
    cy, ch = randn(gen, rows, cols), randn(gen, rows, cols)
    y, h, mean, rstd = nv.layer_norm(x, w, b, center=center)
    dx, dw, db = nv.layer_norm_backward(cy, x, w, mean, rstd, dres=ch)

    def value(x, w, b):
        return ((forward_reference(x, w, b, 1e-5, center)[0] * cy.double()).sum()
                + (x * ch.double()).sum())
    xd, wd, bd = x.double(), w.double(), b.double()
    for _ in range(3):
        for grad, at in ((dx, 0), (dw, 1), (db, 2)):
            v = randn(gen, *grad.shape).double()
            args = [xd, wd, bd]
            e = 1e-4
            up, down = list(args), list(args)
            up[at] = args[at] + e * v
            down[at] = args[at] - e * v
            want = (value(*up) - value(*down)) / (2 * e)
            got = (grad.double() * v).sum()
            # the gradient's own error, element by element, is some (steps + 40) u of its terms
            tol = (steps(cols) + 40) * U * 8 * float((grad.double().abs().max() + 1) * v.abs().sum())
            assert abs(float(got - want)) <= tol + 1e-5 * abs(float(want)), (at, float(got), float(want))


def test_strides_offsets_and_shapes(nv):
    """Row strides, starts at any element, more dimensions, outputs given by the caller."""
    gen = torch.Generator("cuda").manual_seed(5)
    for T in (BF, F):
        for cols, stride, start in ((100, 131, 1), (4096, 4097, 3), (513, 513, 5), (8192, 8200, 7)):
            buf = randn(gen, 9 * stride + 16).to(T)
            x = buf[start:start + 8 * stride].view(8, stride)[:, :cols]
            res = randn(gen, 8 * (stride + 2) + 3).to(T)[1:1 + 8 * (stride + 2)].view(8, stride + 2)[:, :cols]
            w = randn(gen, cols + 1).to(T)[1:]
            b = randn(gen, cols + 3).to(T)[3:]
            yb = torch.full((8 * cols + 32,), 7.0, device="cuda", dtype=T)
            y = yb[9:9 + 8 * cols].view(8, cols)
            check_forward(nv, x, res, w, b, True, y=y)
            assert (yb[:9] == 7).all() and (yb[9 + 8 * cols:] == 7).all()
            check_forward(nv, x, None, w, b, False)
    x = randn(gen, 2, 3, 4, 72)
    w = randn(gen, 72)
    y, _, mean, rstd = nv.layer_norm(x, w)
    assert y.shape == x.shape and mean.shape == rstd.shape == (2, 3, 4)
    flat = nv.layer_norm(x.view(-1, 72), w)[0]
    assert torch.equal(y.view(-1, 72), flat)
    dx, _, _ = nv.layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == x.shape


@pytest.mark.parametrize("T", [BF, F], ids=str)
@pytest.mark.parametrize("cols", [72, 1000, 4096, 4099, 16384, 20001])
def test_in_place(nv, cols, T):
    x, r, w, b, gen = inputs(33, cols, T, T)
    want, h, mean, rstd = nv.layer_norm(x, w, b, residual=r)
    for target in ("x", "residual"):
        a, c = x.clone(), r.clone()
        y, h2, _, _ = nv.layer_norm(a, w, b, residual=c, h=a if target == "x" else c)
        assert torch.equal(y, want) and torch.equal(h2, h)
    want = nv.layer_norm(x, w, b)[0]
    a = x.clone()
    assert torch.equal(nv.layer_norm(a, w, b, y=a)[0], want)
    dy = (randn(gen, 33, cols) * 0.1).to(T)
    dx, dw, db = nv.layer_norm_backward(dy, h, w, mean, rstd, dres=r)
    for target in ("dy", "dres"):
        a, c = dy.clone(), r.clone()
        got = nv.layer_norm_backward(a, h, w, mean, rstd, dres=c, dx=a if target == "dy" else c)
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)


def test_no_rows(nv):
    w = torch.ones(64, device="cuda", dtype=BF)
    x = torch.empty(0, 64, device="cuda", dtype=BF)
    amax = torch.full((1,), 3.0, device="cuda")
    y, _, mean, rstd = nv.layer_norm(x, w, amax=amax)
    assert y.shape == (0, 64) and mean.shape == (0,) and amax.item() == 0.0
    dx, dw, db = nv.layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_values_at_the_edges(nv):
    """A constant row (variance 0), zero rows with eps 0, huge values, NaN and infinity in one
    row: the others stay as they are, and the maximum tells."""
    w = torch.ones(256, device="cuda")
    x = torch.full((3, 256), 3.0, device="cuda")
    y, _, mean, rstd = nv.layer_norm(x, w, eps=1e-5)
    assert (y == 0).all() and (mean == 3).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
    y, _, _, rstd = nv.layer_norm(torch.zeros(2, 256, device="cuda"), w, eps=0.0)
    assert torch.isinf(rstd).all() and torch.isnan(y).all()      # 0 * inf, as the formula says
    gen = torch.Generator("cuda").manual_seed(3)
    x = randn(gen, 4, 256)
    clean = nv.layer_norm(x, w)[0]
    for bad in (float("nan"), float("inf")):
        z = x.clone()
        z[2, 17] = bad
        amax = torch.zeros(1, device="cuda")
        y = nv.layer_norm(z, w, amax=amax)[0]
        assert torch.isnan(y[2]).all() and torch.equal(y[[0, 1, 3]], clean[[0, 1, 3]])
        assert torch.isnan(amax).all()
    big = (x * 1e17)
    check_forward(nv, big, None, w, None, True)


def test_amax_serves_the_quantization(nv):
    """The maximum is nvfp4_amax's, so the fixed-scale calls give the dynamic calls' bits."""
    x, r, w, b, _ = inputs(96, 4096, BF, BF)
    amax = torch.empty(1, device="cuda")
    y = nv.layer_norm(x, w, b, residual=r, amax=amax)[0]
    assert torch.equal(amax, nv.amax(y))
    a, alpha = nv.fakequant(y, "four_over_six", "mae")
    c, alpha2 = nv.fakequant_from_amax(y, amax, "four_over_six", "mae")
    assert torch.equal(a.view(torch.int16), c.view(torch.int16)) and torch.equal(alpha, alpha2)


def test_same_bits_again_and_on_another_stream(nv):
    x, r, w, b, gen = inputs(777, 4096, BF, BF)
    dy = randn(gen, 777, 4096).to(BF)

    def work():
        y, h, mean, rstd = nv.layer_norm(x, w, b, residual=r)
        return (y, h, mean, rstd) + nv.layer_norm_backward(dy, h, w, mean, rstd, dres=r)
    first = work()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = work()
    side.synchronize()
    for p, q in zip(first, second):
        assert torch.equal(p, q)


def test_graph_replays(nv):
    x, r, w, b, gen = inputs(130, 2048, BF, BF)
    dy = randn(gen, 130, 2048).to(BF)
    amax = torch.zeros(1, device="cuda")
    outs = [torch.empty_like(x), torch.empty_like(x), torch.empty(130, device="cuda"),
            torch.empty(130, device="cuda"), torch.empty_like(x), torch.empty_like(w),
            torch.empty_like(w), amax]
    ws = torch.empty(nv.lib().nvfp4_layernorm_backward_workspace(130, 2048), dtype=torch.uint8,
                     device="cuda")

    def work():
        nv.layer_norm(x, w, b, residual=r, y=outs[0], h=outs[1], mean=outs[2], rstd=outs[3], amax=amax)
        nv.layer_norm_backward(dy, outs[1], w, outs[2], outs[3], dx=outs[4], dweight=outs[5],
                               dbias=outs[6], workspace=ws)
    work()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for turn in range(4):
        for t in outs:
            t.fill_(9.0)
        nv.layer_norm(r, w, b)                      # other work between the replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k, (t, e) in enumerate(zip(outs, want)):
            assert torch.equal(t, e), (turn, k)


def test_refusals(nv):
    x, r, w, b, _ = inputs(4, 64, BF, BF)
    m = torch.zeros(4, device="cuda")
    for err, call in (
            (TypeError, lambda: nv.layer_norm(x.half(), w)),
            (TypeError, lambda: nv.layer_norm(x, w.half())),
            (TypeError, lambda: nv.layer_norm(x, w, b.float())),
            (TypeError, lambda: nv.layer_norm(x, w, residual=r.float())),
            (ValueError, lambda: nv.layer_norm(x, w[:63])),
            (ValueError, lambda: nv.layer_norm(x, w, residual=r[:3])),
            (ValueError, lambda: nv.layer_norm(x.t(), torch.ones(4, device="cuda", dtype=BF))),
            (ValueError, lambda: nv.layer_norm(x.expand(2, 4, 64), w)),
            (ValueError, lambda: nv.layer_norm(x, w, h=r)),
            (ValueError, lambda: nv.layer_norm(x, w, amax=m)),
            (ValueError, lambda: nv.layer_norm(x, w.cpu())),
            (nv.NVFP4Error, lambda: nv.layer_norm(x, w, eps=-1.0)),
            (nv.NVFP4Error, lambda: nv.layer_norm(x, w, residual=r, y=x)),
            (ValueError, lambda: nv.layer_norm_backward(x, r[:3], w, m, m)),
            (ValueError, lambda: nv.layer_norm_backward(x, r, w, m[:3], m)),
            (TypeError, lambda: nv.layer_norm_backward(x, r, w, m.double(), m)),
            (ValueError, lambda: nv.layer_norm_backward(
                x, r, w, m, m, workspace=torch.empty(8, device="cuda"))),
            (nv.NVFP4Error, lambda: nv.layer_norm_backward(x, r, w, m, m, dx=r))):
        with pytest.raises(err):
            call()


@pytest.mark.parametrize("T,W", [(BF, BF), (BF, F), (F, F), (F, BF)], ids=str)
@pytest.mark.parametrize("cols", [3, 6, 60, 100, 127, 128, 129, 200, 252, 256, 257])
def test_several_rows_to_a_wavefront(nv, cols, T, W):
    """Rows of a head's width and less, more of them than the workgroups take at a time, their
    number odd; in place, and with strides."""
    for rows in (1, 19, 40013):
        say("[norm] narrow", rows, cols, T, W)
        x, r, w, b, gen = inputs(rows, cols, T, W)
        y, h, mean, rstd = check_forward(nv, x, r, w, b, True)
        a = r.clone()
        again = nv.layer_norm(x, w, b, residual=a, h=a)
        assert torch.equal(again[0], y) and torch.equal(a, h)
        wide = torch.full((rows, cols + 5), 9.0, device="cuda", dtype=T)
        wide[:, :cols] = x
        check_forward(nv, wide[:, :cols], None, w, None, False)
        dy = (0.01 * randn(gen, rows, cols)).to(T)
        dres = (0.01 * r.float()).to(T)
        dx, dw, db = check_backward(nv, dy, h, w, mean, rstd, dres)
        a = dy.clone()
        again = nv.layer_norm_backward(a, h, w, mean, rstd, dres=dres, dx=a)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and torch.equal(again[2], db)
        check_backward(nv, dy, h, w, None, rstd, None, bias=False)


def test_backward_of_a_row_past_a_launch(nv):
    """A row with more columns than one launch has threads for their sums (2^32 / 16)."""
    cols = (1 << 28) + 9
    gen = torch.Generator("cuda").manual_seed(8)
    h, dy = (torch.randn(1, cols, generator=gen, device="cuda", dtype=BF) for _ in range(2))
    w = torch.ones(cols, device="cuda", dtype=BF)
    mean, rstd = torch.full((1,), 0.25, device="cuda"), torch.full((1,), 0.5, device="cuda")
    dx, dw, db = nv.layer_norm_backward(dy, h, w, mean, rstd)
    assert torch.equal(db, dy[0])
    for at in (0, (1 << 26) - 5, (1 << 28) - 100, cols - 50):
        part = slice(at, min(at + 1000, cols))
        want = dy[0, part].double() * (h[0, part].double() - 0.25) * 0.5
        near(dw[part], want, (HALF[BF] + 4 * U) * want.abs() * (1 + HALF[BF])
             + dy[0, part].double().abs() * h[0, part].double().abs() * U + 1e-40, "dweight")


def test_offsets_past_32_bits(nv):
    """More than 2^31 elements: the last rows are what they are by themselves, and the column sums
    have their part."""
    for rows, cols in ((131080, 16384), (8388700, 257)):
        say("[norm] offsets", rows, cols)
        gen = torch.Generator("cuda").manual_seed(4)
        x = torch.zeros(rows, cols, device="cuda", dtype=BF)
        last = randn(gen, 40, cols).to(BF)
        x[-40:] = last
        w, b = randn(gen, cols), randn(gen, cols)
        y, _, mean, rstd = nv.layer_norm(x, w, b)
        y2, _, mean2, rstd2 = nv.layer_norm(last, w, b)
        assert torch.equal(y[-40:], y2) and torch.equal(mean[-40:], mean2) and torch.equal(rstd[-40:], rstd2)
        assert torch.equal(y[:9], b.to(BF).expand(9, cols)) and torch.equal(y[-49:-40], y[:9])
        dy = y.zero_()
        dy[-40:] = randn(gen, 40, cols).to(BF)
        few = dy[-40:].clone()
        dx, dw, db = nv.layer_norm_backward(dy, x, w, mean, rstd)
        want, want_w, want_b, _, xh, _, _ = backward_reference(few, last, w, mean2, rstd2, None)
        dx2, _, _ = check_backward(nv, few, last, w, mean2, rstd2, None)
        assert torch.equal(dx[-40:], dx2) and not dx[:9].any() and not dx[-49:-40].any()
        lever = (few.double().abs() * rstd2.double()[:, None] * last.double().abs() * U).sum(0)
        near(dw, want_w, 104 * U * (few.double() * xh).abs().sum(0) + lever + U * want_w.abs() + 1e-40, "dweight")
        near(db, want_b, 104 * U * few.double().abs().sum(0) + U * want_b.abs() + 1e-40, "dbias")
        del x, y, dy, dx
        torch.cuda.empty_cache()


@pytest.mark.parametrize("T,W", [(BF, BF), (BF, F), (F, F), (F, BF)], ids=str)
@pytest.mark.parametrize("cols", [513, 520, 777, 1016, 1023, 1024, 1025])
def test_backward_of_rows_about_a_wavefronts_length(nv, cols, T, W):
    """Few rows, some hundred, and more than the workgroups take at a time; in place."""
    for rows in (1, 19, 300, 9001):
        h, dres, w, _, gen = inputs(rows, cols, T, W)
        dy = (0.01 * randn(gen, rows, cols)).to(T)
        dres = (0.01 * dres.float()).to(T)
        _, mean, rstd = forward_reference(h, w, None, 1e-5, True)
        mean, rstd = mean[:, 0].float(), rstd[:, 0].float()
        check_backward(nv, dy, h, w, None, rstd, None, bias=False)
        dx, dw, db = check_backward(nv, dy, h, w, mean, rstd, dres)
        for target in ("dy", "dres"):
            a, c = dy.clone(), dres.clone()
            got = nv.layer_norm_backward(a, h, w, mean, rstd, dres=c, dx=a if target == "dy" else c)
            assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)


@pytest.mark.parametrize("T,W", [(BF, BF), (BF, F), (F, F), (F, BF)], ids=str)
@pytest.mark.parametrize("cols", [1032, 1500, 4099, 4104, 6001, 8191, 8200, 14341, 16383])
def test_in_place_of_rows_that_do_not_fill_a_workgroup(nv, cols, T, W):
    """dx over dy and over dres, where a lane past the row's end has its neighbours' elements: more rows
    than workgroups, the same bits as in memory of their own."""
    rows = 1203
    say("[norm] in place", rows, cols, T, W)
    h, dres, w, _, gen = inputs(rows, cols, T, W)
    dy = (0.01 * randn(gen, rows, cols)).to(T)
    _, mean, rstd = forward_reference(h, w, None, 1e-5, True)
    mean, rstd = mean[:, 0].float(), rstd[:, 0].float()
    want = nv.layer_norm_backward(dy, h, w, mean, rstd, dres=dres)
    for target in ("dy", "dres"):
        for _ in range(3):
            a, c = dy.clone(), dres.clone()
            got = nv.layer_norm_backward(a, h, w, mean, rstd, dres=c, dx=a if target == "dy" else c)
            assert all(torch.equal(p, q) for p, q in zip(got, want)), target


class Guarded:
    """Tensors in memory of their own with 64 bytes around them that nothing may write, starting
    `skew` elements into it."""

    def __init__(self):
        self.bufs = []

    def __call__(self, values, skew):
        esize, n = values.element_size(), values.numel()
        buf = torch.full((n * esize + 128 + 16,), 0x5A, device="cuda", dtype=torch.uint8)
        at = 64 + skew * esize
        self.bufs.append((buf, at, at + n * esize))
        part = buf[at:at + n * esize].view(values.dtype).view(values.shape)
        part.copy_(values)
        return part

    def untouched(self):
        return all((b[:lo] == 0x5A).all() and (b[hi:] == 0x5A).all() for b, lo, hi in self.bufs)


@pytest.mark.parametrize("T,W", [(BF, BF), (BF, F), (F, F), (F, BF)], ids=str)
@pytest.mark.parametrize("cols", [5, 100, 200, 513, 1023, 1030, 4099, 8200, 12001, 16383, 20001])
def test_any_start_and_nothing_written_around(nv, cols, T, W):
    """Every operand of both directions at odd starts, the outputs and a workspace of the exact size
    with guards around them: the bits of the aligned call, and the guards as they were."""
    for rows in (1, 6, 301):
        say("[norm] guards", rows, cols, T, W)
        x, r, w, b, gen = inputs(rows, cols, T, W)
        dy = (0.01 * randn(gen, rows, cols)).to(T)
        stat = torch.zeros(rows, device="cuda")
        for res in (None, r):
            for center in (True, False):
                amax = torch.zeros(1, device="cuda")
                want = nv.layer_norm(x, w, b, residual=res, center=center, amax=amax)
                g = Guarded()
                top = g(torch.zeros(1, device="cuda"), 1)
                got = nv.layer_norm(
                    g(x, 1), g(w, 3), g(b, 1), residual=None if res is None else g(res, 3), center=center,
                    amax=top, y=g(torch.zeros_like(x), 1), h=None if res is None else g(torch.zeros_like(x), 3),
                    mean=g(stat, 1) if center else None, rstd=g(stat, 3))
                _, h, mean, rstd = want
                for p, q in zip(got, want):
                    assert (p is None and q is None) or torch.equal(p, q)
                assert torch.equal(top, amax) and g.untouched()
                want = nv.layer_norm_backward(dy, h, w, mean, rstd, dres=res, bias=center)
                g = Guarded()
                work = torch.zeros(nv.lib().nvfp4_layernorm_backward_workspace(rows, cols), device="cuda",
                                   dtype=torch.uint8)
                got = nv.layer_norm_backward(
                    g(dy, 1), g(h, 3), g(w, 1), None if mean is None else g(mean, 1), g(rstd, 3),
                    dres=None if res is None else g(res, 1), bias=center, dx=g(torch.zeros_like(dy), 3),
                    dweight=g(torch.zeros_like(w), 1), dbias=g(torch.zeros_like(w), 3) if center else None,
                    workspace=g(work, 0))
                for p, q in zip(got, want):
                    assert (p is None and q is None) or torch.equal(p, q)
                assert g.untouched()
