"""The distillation loss and its gradient on the GPU against the definition in 64 bits.

Tolerances.  u = 2^-24.  Probabilities: the exponent y = (x - max) c - log2 Z (binary logarithms)
is off by u of its three parts, Z by the s = 16 * ceil(V / 8192) + 64 additions behind it, and
each power of two by one step (2u); together a relative error of e = u (4 + s + 3 (|x - max| c +
log2 Z)).  The gradient is (w / T) (q - p) with these errors and its own rounding.  The loss is a
sum of q - p + p d (d = log p - log q), in which a common error of log Z or of the exponents
cancels against p d: what stays are the steps of the powers of two, 2u (q + p) each, e of |q - p|
and of p |d|, and the additions, s u of the same.
"""
from __future__ import annotations

import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {T: torch.finfo(T).eps / 2 for T in (torch.bfloat16, torch.float32)}     # 2^-8, 2^-24
BF, F = torch.bfloat16, torch.float32
INF = math.inf


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


def logits(rows, vocab, S, T, seed=0, near=0.3, size=2.5):
    gen = torch.Generator("cuda").manual_seed(seed + 31 * rows + vocab)
    t = torch.randn(rows, vocab, generator=gen, device="cuda") * size
    s = t + near * torch.randn(rows, vocab, generator=gen, device="cuda")
    return s.to(S), t.to(T)


def reference(s, t, w, T):
    """loss, gradient, and the tolerances of both."""
    # less the row's largest: next to 1e38, 64 bits have no room for the logarithm of the sum
    s, t = ((x.double() - x.double().amax(1, keepdim=True)) / T for x in (s, t))
    w = torch.ones(s.shape[0], dtype=torch.float64, device="cuda") if w is None else w.double()
    ls, lt = s.logsumexp(1, keepdim=True), t.logsumexp(1, keepdim=True)
    lq, lp = s - ls, t - lt
    q, p = lq.exp(), lp.exp()
    d = torch.where(p > 0, lp - lq, 0.0)
    loss = (p * d).sum(1)
    steps = 16 * -(-s.shape[1] // 8192) + 64
    def rel(x, l):
        top = x.amax(1, keepdim=True)
        far = torch.where(x > -INF, top - x, 0.0) / math.log(2)
        return U * (4 + steps + 3 * (far + (l - top).abs() / math.log(2)))
    # probabilities below 2^-126 come out as 0
    tol_grad = q * rel(s, ls) + p * rel(t, lt) + 2.0 ** -125
    flat, bent = (q - p).abs(), p * d.abs()
    tol_loss = (4 * U * (q + p) + flat * rel(s, ls) + bent * rel(t, lt)
                + steps * U * (flat + bent)).sum(1) + 4 * U * loss.abs()
    grad = (q - p) * (w / T)[:, None]
    return w * loss, grad, tol_loss * w.abs(), tol_grad * (w.abs() / T)[:, None] + 4 * U * grad.abs()


def check(nv, s, t, w=None, T=1.0, **kw):
    want_loss, want_grad, tol_loss, tol_grad = reference(s, t, w, T)
    S = s.dtype
    loss, grad = nv.distill_loss(s, t, w, temperature=T, **kw)
    off = (loss.double() - want_loss).abs()
    assert (off <= tol_loss + 1e-38).all(), ("loss", float((off / (tol_loss + 1e-38)).max()))
    off = (grad.double() - want_grad).abs()
    tol = tol_grad * (1 + HALF[S]) + HALF[S] * want_grad.abs() + 2.0 ** -126
    assert (off <= tol).all(), ("grad", float((off / tol).max()))
    return loss, grad


SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (1, 1000), (7, 8191), (2, 8192), (3, 16384),
         (1, 16385), (2, 32769), (5, 50251), (1, 200001), (200, 1000), (191, 20000), (192, 20000),
         (300, 4099), (1100, 513)]


@pytest.mark.parametrize("S,T", [(BF, BF), (F, F), (BF, F), (F, BF)], ids=str)
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_loss_and_gradient(nv, rows, vocab, S, T):
    say("[distill]", rows, vocab, S, T)
    s, t = logits(rows, vocab, S, T)
    loss, grad = check(nv, s, t)
    gen = torch.Generator("cuda").manual_seed(1)
    w = torch.rand(rows, generator=gen, device="cuda") + 0.1
    w[::3] = 0
    for temp in (2.0, 0.5):
        loss, grad = check(nv, s, t, w, temp)
        assert (loss[::3] == 0).all() and (grad[::3] == 0).all()
    again = nv.distill_loss(s, t, w, temperature=0.5)
    assert torch.equal(again[0], loss) and torch.equal(again[1], grad)
    only, none = nv.distill_loss(s, t, w, temperature=0.5, want_grad=False)
    assert none is None and torch.equal(only, loss)


@pytest.mark.parametrize("rows", [2, 250])
def test_near_and_far_students(nv, rows):
    """A student very close to its teacher keeps its relative precision; one far away, and
    logits of a thousand, stay finite."""
    for near, size in ((0.01, 2.5), (0.1, 2.5), (5.0, 5.0), (0.3, 1000.0)):
        s, t = logits(rows, 20011, F, F, near=near, size=size)
        check(nv, s, t)
    s, t = logits(rows, 20011, F, F, near=0.01)
    loss, _ = nv.distill_loss(s, t)
    want = reference(s, t, None, 1.0)[0]              # about 5e-5, where 8u + ... is 6e-7
    assert ((loss.double() - want).abs() <= 0.02 * want).all()
    loss, grad = nv.distill_loss(t, t)
    assert (loss.abs() <= 64 * U).all() and (grad == 0).all()


@pytest.mark.parametrize("rows,vocab", [(3, 40000), (260, 3001)])
def test_masked_vocabulary_and_rows(nv, rows, vocab):
    """-inf in both (padding), the type's lowest value as a mask, rows of weight 0 full of NaN."""
    for S in (BF, F):
        s, t = logits(rows, vocab, S, S)
        cols = torch.randperm(vocab, generator=torch.Generator().manual_seed(2))[:vocab // 5].cuda()
        s[:, cols] = -INF
        t[:, cols] = -INF
        s[:, -11:] = -INF
        t[:, -11:] = -INF
        w = torch.ones(rows, device="cuda")
        w[1] = 0
        loss, grad = check(nv, s, t, w)
        assert (grad[:, cols] == 0).all()
        s2, t2 = s.clone(), t.clone()
        s2[1] = float("nan")
        t2[1] = INF
        loss2, grad2 = nv.distill_loss(s2, t2, w)
        assert torch.equal(loss2, loss) and torch.equal(grad2, grad)
        low = torch.finfo(S).min
        loss3, grad3 = nv.distill_loss(s.masked_fill(s == -INF, low), t.masked_fill(t == -INF, low), w)
        assert torch.equal(loss3, loss) and torch.equal(grad3, grad)
        # a row in which every entry is the lowest value is uniform, in both: no loss
        s4 = torch.full((rows, vocab), low, device="cuda", dtype=S)
        loss4, grad4 = nv.distill_loss(s4, s4)
        assert (loss4.abs() <= 64 * U).all() and (grad4 == 0).all()
        # only the student excludes an entry that the teacher expects
        s5 = s.clone()
        at = int(t[0].float().argmax())
        s5[0, at] = -INF
        loss5, grad5 = nv.distill_loss(s5, t, w)
        assert loss5[0] == INF and torch.isfinite(grad5[0]).all()
        assert torch.equal(loss5[2:], loss[2:]) and torch.equal(grad5[2:], grad[2:])
        # only the teacher excludes entries: they pull the student down
        t6 = t.clone()
        t6[0, :100] = -INF
        check(nv, s, t6, w)


@pytest.mark.parametrize("rows,vocab", [(2, 40000), (260, 3001)])
@pytest.mark.parametrize("which", ["student", "teacher"])
def test_rows_without_a_distribution(nv, rows, vocab, which):
    s, t = logits(rows, vocab, BF, BF)
    loss, grad = nv.distill_loss(s, t)
    for bad in ("nan", "inf", "empty"):
        s2, t2 = s.clone(), t.clone()
        x = s2 if which == "student" else t2
        if bad == "empty":
            x[0] = -INF
        else:
            x[0, vocab - 1] = float(bad)
        loss2, grad2 = nv.distill_loss(s2, t2)
        assert torch.isnan(loss2[0]) and torch.isnan(grad2[0]).all(), bad
        assert torch.equal(loss2[1:], loss[1:]) and torch.equal(grad2[1:], grad[1:])


@pytest.mark.parametrize("rows,vocab", [(3, 30011), (220, 1003)])
def test_strides_offsets_and_in_place(nv, rows, vocab):
    for S in (BF, F):
        s, t = logits(rows, vocab, S, S)
        loss, grad = nv.distill_loss(s, t)
        sb = torch.zeros(rows * (vocab + 5) + 8, device="cuda", dtype=S)
        sv = sb[3:3 + rows * (vocab + 5)].view(rows, vocab + 5)[:, :vocab]
        sv.copy_(s)
        tb = torch.zeros(rows * (vocab + 9) + 8, device="cuda", dtype=S)
        tv = tb[1:1 + rows * (vocab + 9)].view(rows, vocab + 9)[:, :vocab]
        tv.copy_(t)
        gb = torch.full((rows * (vocab + 3) + 8,), 5.0, device="cuda", dtype=S)
        whole = gb[5:5 + rows * (vocab + 3)].view(rows, vocab + 3)
        loss2, grad2 = nv.distill_loss(sv, tv, grad=whole[:, :vocab])
        assert torch.equal(loss2, loss) and torch.equal(grad2, grad)
        assert (whole[:, vocab:] == 5).all() and (gb[:5] == 5).all() and (gb[5 + whole.numel():] == 5).all()
        loss3, grad3 = nv.distill_loss(sv, tv, grad=sv)
        assert torch.equal(loss3, loss) and torch.equal(sv, grad) and grad3.data_ptr() == sv.data_ptr()
        a = s.clone()
        nv.distill_loss(a, t, grad=a)
        assert torch.equal(a, grad)
    s3 = s[:rows // 2 * 2].view(2, -1, vocab)
    loss4, grad4 = nv.distill_loss(s3, t[:rows // 2 * 2].view(2, -1, vocab))
    assert loss4.shape == s3.shape[:2] and grad4.shape == s3.shape


@pytest.mark.parametrize("vocab", [5, 1000, 30000])
def test_gradient_against_differences(nv, vocab):
    """Differences of the 64-bit loss along random directions.  Step 1e-4: the differences' own
    error is 1e-8 of third derivatives that are below 1."""
    s, t = logits(4, vocab, F, F)
    w = torch.tensor([0.7, 1.0, 0.0, 2.5], device="cuda")
    for T in (1.0, 3.0):
        _, grad = nv.distill_loss(s, t, w, temperature=T)
        gen = torch.Generator("cuda").manual_seed(9)
        for _ in range(3):
            v = torch.randn(4, vocab, generator=gen, device="cuda").double()
            e = 1e-4
            want = (reference(s.double() + e * v, t, w, T)[0] - reference(s.double() - e * v, t, w, T)[0]) / (2 * e)
            got = (grad.double() * v).sum(1)
            tol = (reference(s, t, w, T)[3] * v.abs()).sum(1) + 1e-6
            assert ((got - want).abs() <= tol).all(), (got, want)


def test_no_rows_and_streams(nv):
    e = torch.empty(0, 100, device="cuda")
    loss, grad = nv.distill_loss(e, e)
    assert loss.shape == (0,) and grad.shape == (0, 100)
    for rows, vocab in ((2, 100000), (400, 5000)):
        s, t = logits(rows, vocab, BF, BF)
        first = nv.distill_loss(s, t)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            second = nv.distill_loss(s, t)
        side.synchronize()
        assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])


@pytest.mark.parametrize("rows,vocab", [(2, 60000), (300, 3000)])
def test_graph_replays(nv, rows, vocab):
    s, t = logits(rows, vocab, BF, BF)
    loss, grad = torch.empty(rows, device="cuda"), torch.empty_like(s)
    ws = torch.full((nv.lib().nvfp4_distill_loss_workspace(rows, vocab) + 16,), 255, dtype=torch.uint8,
                    device="cuda")
    work = lambda: nv.distill_loss(s, t, loss=loss, grad=grad, workspace=ws)
    work()
    torch.cuda.synchronize()
    want = loss.clone(), grad.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for turn in range(4):
        loss.fill_(3)
        grad.fill_(3)
        ws.fill_(turn)
        nv.distill_loss(t, s)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[0]) and torch.equal(grad, want[1]), turn


def test_offsets_past_32_bits(nv):
    """2^31 elements are passed by the last rows of a large batch with a wide row stride."""
    vocab, stride, rows = 1000, 12_000_000, 200
    buf = torch.empty(rows * stride, device="cuda", dtype=BF)
    s, t = logits(rows, vocab, BF, BF)
    view = buf.view(rows, stride)[:, :vocab]
    view.copy_(s)
    loss, grad = nv.distill_loss(view, t)
    want = nv.distill_loss(s, t)
    assert torch.equal(loss, want[0]) and torch.equal(grad, want[1])
    y = nv.layer_norm(view, torch.ones(vocab, device="cuda", dtype=BF))[0]
    assert torch.equal(y, nv.layer_norm(s, torch.ones(vocab, device="cuda", dtype=BF))[0])


def test_refusals(nv):
    s, t = logits(4, 100, BF, BF)
    w = torch.ones(4, device="cuda")
    for err, call in (
            (TypeError, lambda: nv.distill_loss(s.half(), t)),
            (TypeError, lambda: nv.distill_loss(s, t.half())),
            (ValueError, lambda: nv.distill_loss(s, t[:, :99])),
            (ValueError, lambda: nv.distill_loss(s, t.cpu())),
            (ValueError, lambda: nv.distill_loss(s, t, w[:3])),
            (TypeError, lambda: nv.distill_loss(s, t, w.double())),
            (ValueError, lambda: nv.distill_loss(s, t, want_grad=False, grad=s)),
            (TypeError, lambda: nv.distill_loss(s, t, grad=s.float())),
            (ValueError, lambda: nv.distill_loss(s.t(), t.t())),
            (nv.NVFP4Error, lambda: nv.distill_loss(s, t, temperature=0.0)),
            (nv.NVFP4Error, lambda: nv.distill_loss(s, t, grad=t))):
        with pytest.raises(err):
            call()


@pytest.mark.parametrize("S,T", [(BF, BF), (F, F), (BF, F), (F, BF)], ids=str)
@pytest.mark.parametrize("vocab", [9001, 20003, 40008, 70001, 100003, 150001])
def test_rows_of_every_held_length(nv, vocab, S, T):
    """One workgroup to a row, with what it holds of the row filled, passed, and cut: from rows in
    registers alone to ones of which a part is read again.  Also the rows that are done with exact
    differences, at these lengths."""
    say("[distill]", 192, vocab, S, T)
    s, t = logits(192, vocab, S, T)
    s[7, ::5] = -INF
    t[7, ::5] = -INF
    s[8] = torch.finfo(S).min
    w = torch.rand(192, generator=torch.Generator("cuda").manual_seed(3), device="cuda") + 0.1
    w[::2] = 0
    w[8] = 1
    loss, grad = check(nv, s, t, w, 0.7)
    again, same = nv.distill_loss(s, t, w, temperature=0.7, grad=s)
    assert torch.equal(again, loss) and torch.equal(same, grad)


@pytest.mark.parametrize("rows,vocab", [(1, 32769), (3, 50011), (100, 40009), (127, 33000)])
def test_rows_of_several_workgroups(nv, rows, vocab):
    """Few long rows, which several workgroups share, and the same rows among many, which have one
    each: both hold to the definition."""
    for S, T in ((BF, BF), (F, F), (BF, F)):
        s, t = logits(rows, vocab, S, T, near=0.01)
        check(nv, s, t)
        many = [torch.cat([x, x[:1].expand(128 - rows, vocab)]).contiguous() for x in (s, t)]
        check(nv, *many)
        s, t = logits(rows, vocab, S, T, near=5.0, size=1000.0)
        check(nv, s, t)
        s[0] = torch.finfo(S).min
        check(nv, s, t)
    if rows < 100:
        test_strides_offsets_and_in_place(nv, max(rows, 2), vocab)
    test_gradient_against_differences(nv, vocab)


@pytest.mark.parametrize("rows,vocab", [(3, 5), (200, 2000), (2, 40000)])
def test_large_logits(nv, rows, vocab):
    """Logits (over T) so large that a 32-bit exponent has few bits left, or none, for the logarithm
    of the sum."""
    for S, T in ((F, F), (BF, F), (BF, BF)):
        for size, temp in ((100.0, 0.01), (100.0, 0.001), (2e4, 1.0), (1e6, 1.0), (1e10, 1.0), (1e30, 3.0)):
            say("[distill] large", rows, vocab, S, T, size, temp)
            s, t = logits(rows, vocab, S, T, near=0.3, size=size)
            s[0, 1] = t[0, 1] = s[0, 0]           # shared largest entries, in some rows
            s[0, 2], t[0, 2] = s[0, 0], s[0, 0]
            check(nv, s, t, T=temp)
            check(nv, t.to(S), t, T=temp)
            check(nv, s * 0.0, t, T=temp)


@pytest.mark.parametrize("S,T", [(BF, BF), (F, F), (BF, F), (F, BF)], ids=str)
@pytest.mark.parametrize("vocab", [11, 512, 513, 1001, 1024, 1025, 2047, 2049, 3001, 4096, 4097, 6007, 8192, 8193])
def test_short_rows(nv, vocab, S, T):
    """Every number of vectors that a thread may hold, filled and not, rows beginning anywhere."""
    say("[distill] short", vocab, S, T)
    s, t = logits(130, vocab, S, T)
    w = torch.rand(130, generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    w[::7] = 0
    loss, grad = check(nv, s, t, w, 1.5)
    buf = torch.zeros(130 * (vocab + 1) + 1, device="cuda", dtype=S)
    view = buf[1:].view(130, vocab + 1)[:, :vocab]
    view.copy_(s)
    again, same = nv.distill_loss(view, t, w, temperature=1.5, grad=view)
    assert torch.equal(again, loss) and torch.equal(same, grad)
    assert not buf[vocab + 1::vocab + 1].any() and buf[0] == 0


@pytest.mark.parametrize("rows,vocab", [(3, 7), (260, 3001), (3, 40000), (130, 60001)])
def test_a_student_masked_by_a_finite_value(nv, rows, vocab):
    """The student excludes, by the type's lowest value or another far below all, an entry that the
    teacher expects: the loss is p (top - mask) / T, a number, not infinity.  Its other parts are no
    part of it in 32 bits, so it is off by the error of p (in the header) and 8 roundings."""
    gen = torch.Generator("cuda").manual_seed(5)
    for S, T in ((BF, BF), (F, F), (BF, F), (F, BF)):
        for size, temp, mask in ((2.5, 1.0, None), (2.5, 2.0, None), (2.5, 0.7, None), (2.5, 1.0, -1e36),
                                 (2.5, 0.01, -1e36), (1e6, 3.0, None), (1e37, 3.0, None)):
            say("[distill] finite mask", rows, vocab, S, T, size, temp, mask)
            s, t = logits(rows, vocab, S, T, size=size, near=0.3 * size)
            top = t.double().amax(1, keepdim=True)
            p = torch.softmax((t.double() - top) / temp, 1)
            # expected by the teacher with at most a quarter: no loss passes the largest number
            at = torch.where(p <= 0.25, p, -1.0).argmax(1)
            each = torch.arange(rows, device="cuda")
            if rows > 100:                        # not the rows of even number: they stay as they are
                each, at = each[1::2], at[1::2]
            clean = s.clone()
            s[each, at] = torch.finfo(S).min if mask is None else mask
            w = torch.rand(rows, generator=gen, device="cuda") + 0.1
            want, want_grad, tol, tol_grad = reference(s, t, w, temp)
            d = (s.double().amax(1)[each] - s.double()[each, at]) / temp
            main = w.double()[each] * p[each, at] * d
            far = (top[each, 0] - t.double()[each, at]) / temp / math.log(2)
            logz = torch.log2(torch.exp((t.double() - top) / temp).sum(1))[each]
            steps = 16 * -(-vocab // 8192) + 64
            rel = U * (4 + steps + 3 * (far + logz)) + 8 * U
            loss, grad = nv.distill_loss(s, t, w, temperature=temp)
            sure = p[each, at] > 2.0 ** -100              # where the teacher's probability is a number
            off = (loss.double()[each] - main).abs() / main.clamp(min=1e-300)
            # what is left out of `main`: the rest of the loss
            rest = (want[each] - main).abs() / main.clamp(min=1e-300)
            assert (off <= rel + rest)[sure].all(), float((off / (rel + rest))[sure].max())
            ok = (grad.double() - want_grad).abs() <= (tol_grad * (1 + HALF[S]) + HALF[S] * want_grad.abs()
                                                       + 2.0 ** -126)
            assert ok.all()
            again, same = nv.distill_loss(s, t, w, temperature=temp, grad=s)
            assert torch.equal(again, loss) and torch.equal(same, grad)
            if rows > 100:
                plain = nv.distill_loss(clean, t, w, temperature=temp)
                assert torch.equal(loss[::2], plain[0][::2]) and torch.equal(grad[::2], plain[1][::2])
