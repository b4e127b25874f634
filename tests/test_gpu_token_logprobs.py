"""Log probabilities of given tokens, entropy, top alternatives and their gradient against 64 bits (GPU).

Tolerances, with u = 2^-24.  d = (x - m) / T carries three roundings of a binary32 operation or constant,
so a term 2^d of Z is off by 3 |d| u and its own power (2 u); a thread adds vocab / 256 terms or fewer one
after the other (vocab / 64 where a wavefront takes a row) and the rest in a tree, each addition u of the
sum.  ln Z is off by as much absolutely as Z is relatively; logp adds the roundings of its own d and of the
result.  In S = sum d 2^d a term's error counts d-fold.  A gradient is p (A y + B) with y = d - z."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_block_scaled_amax_amd as m
    m.lib()
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def logits_of(shape, seed, kind="model"):
    x = torch.randn(shape, generator=gen(seed))
    if kind == "model":
        x *= 2.5
    elif kind == "ties":
        x = (x * 2).round()
    elif kind == "equal":
        x = torch.full(shape, -1.25)
    elif kind == "rising":
        x = torch.arange(shape[-1]).float().expand(shape).clone() / 64
    elif kind == "clumped":                   # a few threads' vectors hold all that is large
        at = torch.arange(shape[-1])
        x += 30.0 * ((at // 8) % 256 < 2)
    elif kind == "large":
        x *= 3e4
    elif kind == "masked":
        x[torch.rand(shape, generator=gen(seed + 1)) < 0.97] = -INF
        x[..., shape[-1] // 2] = 1.0
    elif kind == "lowest":
        x[torch.rand(shape, generator=gen(seed + 1)) < 0.5] = torch.finfo(BF16).min
    elif kind == "allowed":                   # a grammar's few tokens
        x[torch.rand(shape, generator=gen(seed + 1)) < 1 - 7 / shape[-1]] = -INF
        x[..., 3] = 0.5
    elif kind == "stairs":                    # the largest in one thread's vectors, many of them alike
        at = torch.arange(shape[-1])
        x = torch.where((at // 8) % 256 == 17, 8.0, x.round())
    elif kind == "zeros":
        x = torch.where(x > 0, 0.0, -0.0)
    return x


def tokens_of(rows, given, vocab, seed, none=0.0):
    t = torch.randint(0, vocab, (rows, given), generator=gen(seed))
    t[torch.rand(rows, given, generator=gen(seed + 1)) < none] = -1
    return t


def reference(x, tokens, T, top, threads=256):
    """In 64 bits, with the bounds of logp, of entropy and of ln Z."""
    x = x.double().cpu()
    vocab = x.shape[1]
    m = x.amax(1, keepdim=True)
    d = (x - m) / T
    e = d.exp()
    total = e.sum(1, keepdim=True)
    p, z = e / total, total.log()
    far = torch.where(e > 0, d, torch.zeros_like(d))
    n = vocab / threads + 40
    dz = U * (n + 3 * (p * far.abs()).sum(1) + 4)
    h = z[:, 0] - (p * far).sum(1)
    dh = 2 * dz + U * (3 * (p * far * far).sum(1) + (n + 8) * (1 + h))
    t = tokens.clamp(min=0)
    logp = torch.where(tokens >= 0, d.gather(1, t) - z, 0.0)
    order = torch.sort(x + 0.0, dim=1, descending=True, stable=True).indices[:, :top]
    return dict(m=m[:, 0], z=z[:, 0], d=d, p=p, h=h, logp=logp, top=order, top_logp=d.gather(1, order) - z, dz=dz,
                dh=dh)


def near(got, want, bound):
    """Within the bound, and the same infinities."""
    got = got.double().cpu()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])
    off = (got - want)[~inf].abs()
    bound = torch.as_tensor(bound, dtype=torch.float64).expand(want.shape)[~inf]
    assert (off <= bound).all(), (off / bound).max()


def check_forward(nv, x, tokens, T, top, itype=torch.int64, threads=256):
    logp, entropy, top_logp, top_index, stats = nv.token_logprobs(x, tokens.to(itype).cuda(), top=top,
                                                                  temperature=T)
    live = (tokens >= 0).any(1)
    r = reference(x, tokens, T, top, threads)
    bound = lambda v: r["dz"][:, None] + U * (8 * v.abs().nan_to_num(posinf=0.0) + 4 * r["z"][:, None])
    near(logp.cpu()[live], r["logp"][live], bound(r["logp"])[live])
    near(entropy.cpu()[live], r["h"][live], r["dh"][live])
    assert torch.equal(stats.cpu()[live, 0].double(), r["m"][live])
    near(stats.cpu()[live, 1], r["z"][live], (r["dz"] + 2 * U * r["z"])[live])
    assert not logp.cpu()[~live].any() and not entropy.cpu()[~live].any() and not stats.cpu()[~live].any()
    if top:
        assert top_index.dtype == torch.int64
        assert torch.equal(top_index.cpu()[live], r["top"][live])
        near(top_logp.cpu()[live], r["top_logp"][live], bound(r["top_logp"])[live])
        assert (top_index.cpu()[~live] == -1).all() and not top_logp.cpu()[~live].any()
    else:
        assert top_logp is None and top_index is None
    return r


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab,given,top,T", [
    (1, 1, 1, 1, 1.0), (2, 2, 1, 2, 0.5), (3, 7, 3, 7, 1.0), (2, 64, 64, 64, 2.0), (5, 100, 2, 20, 1.0),
    (3, 1000, 1, 0, 0.7), (7, 2047, 20, 64, 1.0), (130, 2048, 1, 5, 1.0), (4, 2049, 1, 64, 1.0),
    (120, 16384, 1, 20, 1.0), (6, 16385, 2, 64, 0.8), (1, 50251, 1, 20, 1.0), (3, 50251, 8, 64, 1.3),
    (101, 32001, 1, 1, 1.0), (1, 128000, 1, 20, 0.8), (9, 131072, 64, 64, 1.0), (64, 20000, 1, 3, 1.0),
    (101, 200003, 1, 20, 1.0)])
def test_forward(nv, rows, vocab, given, top, T, dtype):
    x = logits_of((rows, vocab), vocab + rows).to(dtype).cuda()
    check_forward(nv, x, tokens_of(rows, given, vocab, 3, 0.2), T, top, torch.int32 if rows % 2 else torch.int64)


KINDS = ["ties", "equal", "rising", "clumped", "large", "masked", "lowest", "zeros", "allowed", "stairs"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab,top", [(3, 333, 20), (2, 5000, 64), (120, 33333, 20), (2, 100003, 64)])
def test_forward_of_difficult_rows(nv, rows, vocab, top, dtype, kind):
    x = logits_of((rows, vocab), 5, kind).to(dtype).cuda()
    check_forward(nv, x, tokens_of(rows, 4, vocab, 3), 1.0, top)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab,given,top", [
    (2049, 1, 1, 1), (2100, 7, 2, 7), (2050, 64, 1, 20), (2500, 333, 3, 24), (3001, 2048, 1, 0), (2049, 4095, 1, 24),
    (2049, 8192, 20, 1), (2100, 8193, 1, 20), (2600, 2000, 64, 64)])
def test_many_short_rows(nv, rows, vocab, given, top, dtype):
    x = logits_of((rows, vocab), vocab + rows).to(dtype).cuda()
    check_forward(nv, x, tokens_of(rows, given, vocab, 3, 0.2), 1.0, top, threads=64)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_short_difficult_rows(nv, dtype, kind):
    x = logits_of((2100, 3333), 5, kind).to(dtype).cuda()
    check_forward(nv, x, tokens_of(2100, 4, 3333, 3), 1.0, 20, threads=64)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_short_rows_without_a_distribution(nv, dtype):
    x = logits_of((2304, 1001), 1).to(dtype)
    x[0, 1000], x[1, 0], x[2], x[3, 500], x[4, 3:5], x[5] = NAN, INF, -INF, -NAN, INF, NAN
    got = [v.cpu() for v in nv.token_logprobs(x.cuda(), tokens_of(2304, 2, 1001, 1).cuda(), top=9)]
    for v in (got[0], got[1], got[2], got[4]):
        assert torch.isnan(v[:6]).all() and not torch.isnan(v[6:]).any()
    assert (got[3][:6] == -1).all() and (got[3][6:] >= 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1e-30, 1e-3, 1e4, 1e30])
def test_extreme_temperatures(nv, T, dtype):
    """Of 1e-30: the largest entry alone (ties share), the others at -inf or far below; of 1e30: all alike."""
    x = logits_of((3, 500), 1).to(dtype).cuda()
    t = torch.tensor(T, dtype=F32).item()
    r = check_forward(nv, x, tokens_of(3, 2, 500, 2), t, 5) if T > 1e-20 else None
    if r is None:
        logp, entropy, top_logp, top_index, stats = nv.token_logprobs(x, torch.zeros(3, dtype=torch.int64,
                                                                                   device="cuda"), top=1, temperature=T)
        m = x.float().amax(1, keepdim=True)
        many = (x.float() == m).sum(1).float().log()
        assert torch.allclose(entropy, many, atol=1e-6) and torch.allclose(top_logp[:, 0], -many, atol=1e-6)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab", [(2, 300), (120, 20001), (2, 70001)])
def test_rows_without_a_distribution(nv, rows, vocab, dtype):
    """NaN, +inf, nothing but -inf: NaN and -1 for these rows, nothing for the others, both ways."""
    x = logits_of((rows + 6, vocab), 1).to(dtype)
    x[0, vocab - 1], x[1, 0], x[2], x[3, vocab // 2], x[4, 3:5] = NAN, INF, -INF, -NAN, INF
    x[5] = NAN
    x, t = x.cuda(), tokens_of(rows + 6, 2, vocab, 1)
    got = nv.token_logprobs(x, t.cuda(), top=9)
    logp, entropy, top_logp, top_index, stats = [v.cpu() for v in got]
    for v in (logp, entropy, top_logp, stats):
        assert torch.isnan(v[:6]).all() and not torch.isnan(v[6:]).any()
    assert (top_index[:6] == -1).all() and (top_index[6:] >= 0).all()
    grad = nv.token_logprobs_backward(x, t.cuda(), got[4], torch.ones(rows + 6, 2, device="cuda"))
    assert torch.isnan(grad[:6]).all() and not torch.isnan(grad[6:]).any()
    check_forward(nv, x[6:], t[6:], 1.0, 9)


@pytest.mark.parametrize("rows,vocab", [(4, 100), (4, 40000)])
def test_tokens_that_are_none_or_beyond(nv, rows, vocab):
    x = logits_of((rows, vocab), 1).cuda()
    x[0] = NAN                                # not read
    t = torch.tensor([[-1, -7], [-1, 5], [vocab, 3], [2 ** 40, -2 ** 62]]).cuda()
    logp, entropy, top_logp, top_index, stats = nv.token_logprobs(x, t, top=3)
    assert not logp[0].any() and entropy[0] == 0 and not stats[0].any()
    assert (top_index[0] == -1).all() and not top_logp[0].any()
    want = torch.log_softmax(x.double(), 1)
    assert logp[1, 0] == 0 and abs(logp[1, 1] - want[1, 5]) < 1e-4
    assert torch.isnan(logp[2, 0]) and abs(logp[2, 1] - want[2, 3]) < 1e-4
    assert torch.isnan(logp[3, 0]) and logp[3, 1] == 0
    g = nv.token_logprobs_backward(x, t, stats, torch.ones(rows, 2, device="cuda"))
    assert not g[0].any() and not torch.isnan(g[1]).any() and torch.isnan(g[2:]).all()


@pytest.mark.parametrize("rows,vocab", [(3, 1000), (3, 60000)])
def test_without_tokens_and_leading_dimensions(nv, rows, vocab):
    x = logits_of((2, rows, vocab), 1).to(BF16).cuda()
    logp, entropy, top_logp, top_index, stats = nv.token_logprobs(x, top=4)
    assert logp is None and entropy.shape == (2, rows) and stats.shape == (2, rows, 2)
    assert top_logp.shape == top_index.shape == (2, rows, 4)
    t = tokens_of(2 * rows, 1, vocab, 1).view(2, rows)
    again = nv.token_logprobs(x, t.cuda())
    assert again[0].shape == (2, rows) and torch.equal(again[1], entropy) and torch.equal(again[4], stats)
    g = nv.token_logprobs_backward(x, t.cuda(), stats, torch.ones(2, rows, device="cuda"))
    assert g.shape == x.shape
    one = nv.token_logprobs(x[1, 2], t[1, 2].cuda(), top=4)
    assert one[0].shape == () and torch.equal(one[3], top_index[1, 2])
    assert nv.token_logprobs(x[:0], t[:0].cuda(), top=4)[3].shape == (0, rows, 4)
    assert nv.token_logprobs_backward(x[:0], t[:0].cuda(), stats[:0], torch.ones(0, rows, device="cuda")).numel() == 0


def check_backward(nv, x, tokens, T, seed, entropy=True, grad=None, itype=torch.int64):
    rows, given = tokens.shape
    r = reference(x, tokens, T, 0)
    dlogp = torch.randn(rows, given, generator=gen(seed))
    dh = torch.randn(rows, generator=gen(seed + 1)) if entropy else None
    stats = torch.stack((r["m"], r["z"]), 1).float()
    got = nv.token_logprobs_backward(x, tokens.to(itype).cuda(), stats.cuda(), dlogp.cuda(),
                                     entropy=r["h"].float().cuda() if entropy else None,
                                     dentropy=dh.cuda() if entropy else None, temperature=T, grad=grad)
    assert got.dtype == x.dtype
    g = torch.where(tokens >= 0, dlogp.double(), 0.0)
    all_, h = g.sum(1, keepdim=True), (dh.double()[:, None] if entropy else torch.zeros(rows, 1))
    lp, p = r["d"] - r["z"][:, None], r["p"]
    low = torch.where(p > 0, lp, 0.0)
    hot = torch.zeros_like(p).scatter_add_(1, tokens.clamp(min=0), g)
    size = torch.zeros_like(p).scatter_add_(1, tokens.clamp(min=0), g.abs())
    live = (tokens >= 0).any(1)[:, None]
    want = torch.where(live, (hot - p * (all_ + h * (low + r["h"][:, None]))) / T, 0.0)
    inner = (h * low).abs() + g.abs().sum(1, keepdim=True) + (h * r["h"][:, None]).abs()
    bound = U / T * (p * inner * (5 * low.abs() + 3 * r["z"][:, None] + given + 16) + (given + 4) * size)
    bound = bound * 2 + torch.finfo(x.dtype).eps / 2 * (want.abs() + bound) + 1e-37
    near(got, want, bound)
    return dlogp, dh


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab,given,T", [
    (1, 1, 1, 1.0), (2, 2, 64, 0.5), (3, 7, 3, 1.0), (4, 2047, 20, 2.0), (3, 2048, 1, 1.0), (5, 16384, 1, 1.0),
    (2, 16385, 64, 0.7), (1, 50251, 8, 1.0), (70, 33000, 1, 1.0)])
@pytest.mark.parametrize("entropy", [False, True])
def test_backward(nv, rows, vocab, given, T, dtype, entropy):
    x = logits_of((rows, vocab), vocab + rows).to(dtype).cuda()
    tokens = tokens_of(rows, given, vocab, 3, 0.2)
    if given > 2:
        tokens[0, 0], tokens[0, -1] = vocab - 1, vocab - 1            # the same token twice
    check_backward(nv, x, tokens, T, 4, entropy, itype=torch.int32 if rows % 2 else torch.int64)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_backward_of_difficult_rows(nv, dtype, kind):
    x = logits_of((3, 5000), 5, kind).to(dtype).cuda()
    check_backward(nv, x, tokens_of(3, 4, 5000, 3), 1.0, 2)


def test_backward_against_differences(nv):
    """The whole way: the gradient of sum(dlogp logp) + sum(dentropy entropy), both from this package,
    against central differences of the same sum in 64 bits."""
    rows, vocab, T = 3, 40, 1.3
    x, tokens = logits_of((rows, vocab), 2).cuda(), tokens_of(rows, 3, vocab, 1, 0.3)
    dlogp, dh = torch.randn(rows, 3, generator=gen(5)), torch.randn(rows, generator=gen(6))
    logp, entropy, _, _, stats = nv.token_logprobs(x, tokens.cuda(), temperature=T)
    got = nv.token_logprobs_backward(x, tokens.cuda(), stats, dlogp.cuda(), entropy=entropy, dentropy=dh.cuda(),
                                     temperature=T).cpu()

    def f(v):
        lp = torch.log_softmax(v / T, 1)
        s = torch.where(tokens >= 0, lp.gather(1, tokens.clamp(min=0)) * dlogp, 0.0).sum(1)
        return torch.where((tokens >= 0).any(1), s - dh * (lp.exp() * lp).sum(1), 0.0)
    v = x.double().cpu()
    for j in range(vocab):
        step = torch.zeros_like(v)
        step[:, j] = 1e-5
        want = (f(v + step) - f(v - step)) / 2e-5
        assert (got[:, j] - want).abs().max() < 2e-6


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [777, 33333])
def test_in_place_strides_and_guards(nv, vocab, dtype):
    """grad over the logits; logits and grad with rows apart that start at odd elements, nothing beside them
    written; outputs between guards."""
    rows, tokens = 5, tokens_of(5, 6, vocab, 1, 0.3)
    tokens[1] = -1
    tokens[2, 1] = tokens[2, 4] = 7
    x = logits_of((rows, vocab), 1).to(dtype)
    held = torch.full((rows, vocab + 37), 3.0, dtype=dtype, device="cuda")
    view = held[:, 5:5 + vocab]
    view.copy_(x)
    check_forward(nv, view, tokens, 1.0, 9)
    other = torch.full((rows, vocab + 19), 3.0, dtype=dtype, device="cuda")
    check_backward(nv, view, tokens, 1.0, 2, grad=other[:, 3:3 + vocab])
    assert (other[:, :3] == 3).all() and (other[:, 3 + vocab:] == 3).all()
    assert torch.equal(view.cpu(), x)
    whole = view.clone()
    r = reference(x, tokens, 1.0, 0)
    args = tokens.cuda(), torch.stack((r["m"], r["z"]), 1).float().cuda(), torch.ones(5, 6, device="cuda")
    nv.token_logprobs_backward(view, *args, grad=view)
    assert (held[:, :5] == 3).all() and (held[:, 5 + vocab:] == 3).all()
    assert torch.equal(view, nv.token_logprobs_backward(whole, *args))

    n = rows * 9
    f, i = torch.full((4, 128 + n), 3.0, device="cuda"), torch.full((n + 64,), 3, device="cuda")
    mid = lambda t, *shape: t[32:32 + math.prod(shape)].view(shape)
    need = nv.lib().nvfp4_token_logprobs_workspace(rows, vocab, 9)
    work = torch.full((need + 64,), 9, dtype=torch.uint8, device="cuda")
    nv.token_logprobs(whole, tokens.cuda(), top=9, logp=mid(f[0], rows, 6), entropy=mid(f[1], rows),
                      top_logp=mid(f[2], rows, 9), top_index=mid(i, rows, 9), stats=mid(f[3], rows, 2),
                      workspace=work[32:32 + need] if need else None)
    for row, size in zip(f, (rows * 6, rows, n, rows * 2)):
        assert (row[:32] == 3).all() and (row[32 + size:] == 3).all()
    assert (i[:32] == 3).all() and (i[32 + n:] == 3).all()
    assert (work[:32] == 9).all() and (work[32 + need:] == 9).all()


def test_far_rows(nv):
    """Logits past 2^32 elements."""
    rows, vocab = 70000, 65000
    x = torch.zeros(rows, vocab, dtype=BF16, device="cuda")
    t = torch.zeros(rows, dtype=torch.int64, device="cuda")
    x[-1, 7], x[-1, 9], t[-1] = 3.0, 12.0, 7
    logp, entropy, top_logp, top_index, stats = nv.token_logprobs(x, t, top=2)
    flat = -math.log(vocab)
    last = math.log(vocab - 2 + math.exp(3) + math.exp(12))
    assert (logp[:-1] - flat).abs().max() < 1e-3 and abs(logp[-1].item() - 3 + last) < 1e-4
    assert top_index[-1].tolist() == [9, 7] and top_index[-2].tolist() == [0, 1]
    nv.token_logprobs_backward(x, t, stats, torch.ones(rows, device="cuda"), grad=x)
    assert abs(x[-1, 7].item() - 1 + math.exp(3 - last)) < 0.01 and abs(x[-1, 9].item() + math.exp(12 - last)) < 0.01
    assert abs(x[-2, 0].item() - 1) < 0.01 and abs(x[-2, 1].item() + 1 / vocab) < 1e-6


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab,top", [(3, 5, 5), (2, 777, 20), (3, 20003, 20), (2, 70001, 20), (2100, 1003, 9)])
def test_a_row_where_it_lies(nv, rows, vocab, top, dtype):
    """At every element of 16 bytes: the bits of the aligned rows, forward and backward, whatever the gradient's
    place."""
    x = logits_of((rows, vocab), 8).to(dtype).cuda()
    t = tokens_of(rows, 2, vocab, 1, 0.2).cuda()
    wide = (vocab + 15) // 8 * 8
    even = torch.zeros(rows, wide, dtype=dtype, device="cuda")
    even[:, :vocab] = x
    want = nv.token_logprobs(even[:, :vocab], t, top=top)
    d, h = torch.randn(rows, 2, device="cuda"), torch.randn(rows, device="cuda")
    back = dict(entropy=want[1], dentropy=h)
    grad = nv.token_logprobs_backward(even[:, :vocab], t, want[4], d, **back)
    for shift in range(1, 8):
        held = torch.full((rows, wide + 8), 5.0, dtype=dtype, device="cuda")
        held[:, shift:shift + vocab] = x
        there = held[:, shift:shift + vocab]
        for a, b in zip(nv.token_logprobs(there, t, top=top), want):
            assert torch.equal(a, b)
        assert torch.equal(nv.token_logprobs_backward(there, t, want[4], d, **back), grad)
        out = torch.full((rows, wide + 8), 7.0, dtype=dtype, device="cuda")
        nv.token_logprobs_backward(x, t, want[4], d, **back, grad=out[:, shift:shift + vocab])
        assert torch.equal(out[:, shift:shift + vocab], grad)
        assert (out[:, :shift] == 7).all() and (out[:, shift + vocab:] == 7).all()
        nv.token_logprobs_backward(there, t, want[4], d, **back, grad=there)
        assert torch.equal(there, grad) and (held[:, :shift] == 5).all() and (held[:, shift + vocab:] == 5).all()


@pytest.mark.parametrize("dtype,rows", [(BF16, 1400), (F32, 700)])
def test_a_gradient_that_no_cache_holds(nv, dtype, rows):
    """More than 128 MB at once: the bits of 100 rows at a time."""
    vocab = 50001
    wide = torch.randn(rows, vocab + 6, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(dtype)
    x, t = wide[:, 3:3 + vocab], tokens_of(rows, 3, vocab, 2, 0.5).cuda()
    entropy, stats = nv.token_logprobs(x, t)[1::3]
    d, h = torch.randn(rows, 3, device="cuda"), torch.randn(rows, device="cuda")
    whole = nv.token_logprobs_backward(x, t, stats, d, entropy=entropy, dentropy=h)
    for i in range(0, rows, 100):
        part = slice(i, i + 100)
        got = nv.token_logprobs_backward(x[part], t[part], stats[part], d[part], entropy=entropy[part], dentropy=h[part])
        assert torch.equal(got, whole[part])


@pytest.mark.parametrize("rows,vocab", [(3, 1500), (2, 90000)])
def test_graphs_and_streams(nv, rows, vocab):
    """Both ways captured on a stream of its own, replayed with other logits, eager calls between: the same
    bits as the eager call each time."""
    x, t = torch.zeros(rows, vocab, dtype=BF16, device="cuda"), torch.zeros(rows, 2, dtype=torch.int64, device="cuda")
    up, dh = torch.ones(rows, 2, device="cuda"), torch.ones(rows, device="cuda")

    def both():
        out = nv.token_logprobs(x, t, top=10)
        return out + (nv.token_logprobs_backward(x, t, out[4], up, entropy=out[1], dentropy=dh),)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = both()
    for seed in range(4):
        x.copy_(logits_of((rows, vocab), seed).to(BF16))
        t.copy_(tokens_of(rows, 2, vocab, seed))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, both()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_refusals(nv):
    x, t = torch.zeros(4, 100, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    s, g = torch.zeros(4, 2, device="cuda"), torch.zeros(4, device="cuda")
    f, b = nv.token_logprobs, nv.token_logprobs_backward
    bad = [
        (TypeError, "logits must be", lambda: f(x.double(), t)),
        (ValueError, "contiguous", lambda: f(x.t(), t)),
        (ValueError, "tokens must have shape", lambda: f(x, t[:3])),
        (ValueError, "tokens must have shape", lambda: f(x, t[:, None, None])),
        (TypeError, "tokens must be", lambda: f(x, t.float())),
        (ValueError, "tokens must be on", lambda: f(x, t.cpu())),
        (ValueError, "1 to 64", lambda: f(x, t[:, None].repeat(1, 65))),
        (ValueError, "1 to 64", lambda: f(x, t[:, None][:, :0])),
        (ValueError, "top must be", lambda: f(x, t, top=65)),
        (ValueError, "top must be", lambda: f(x[:, :9], t, top=10)),
        (ValueError, "top must be", lambda: f(x, t, top=-1)),
        (ValueError, "form with tokens", lambda: f(x, logp=g)),
        (ValueError, "form with top", lambda: f(x, t, top_logp=g)),
        (ValueError, "output must be", lambda: f(x, t, logp=s)),
        (nv.NVFP4Error, "outside its range", lambda: f(x, t, temperature=0.0)),
        (nv.NVFP4Error, "outside its range", lambda: f(x, t, temperature=-1.0)),
        (nv.NVFP4Error, "overlap", lambda: f(x, t, entropy=x.view(-1)[:4])),
        (TypeError, "logits must be", lambda: b(x.half(), t, s, g)),
        (ValueError, "stats must have shape", lambda: b(x, t, s[:, 0], g)),
        (ValueError, "dlogp must have shape", lambda: b(x, t, s, s)),
        (TypeError, "dlogp must be", lambda: b(x, t, s, g.double())),
        (ValueError, "dentropy needs", lambda: b(x, t, s, g, dentropy=g)),
        (TypeError, "grad must be", lambda: b(x, t, s, g, grad=x.bfloat16())),
        (nv.NVFP4Error, "overlap", lambda: b(x, t, x.view(-1)[:8].view(4, 2), g, grad=x)),
        (nv.NVFP4Error, "outside its range", lambda: b(x, t, s, g, temperature=float("nan"))),
    ]
    for kind, text, call in bad:
        with pytest.raises(kind, match=text):
            call()


def test_two_streams_at_once(nv):
    """Calls on two streams that overlap, rows shared by several workgroups among them: each has the bits it has alone."""
    cases = [(logits_of(shape, 3).to(dtype).cuda(), tokens_of(shape[0], 2, shape[1], 4).cuda())
             for shape, dtype in (((2, 90001), BF16), ((700, 5003), F32), ((3, 128000), BF16), ((2500, 700), BF16))]
    want = [nv.token_logprobs(x, t, top=20) for x, t in cases]
    d = [torch.ones(t.shape, device="cuda") for _, t in cases]
    grads = [nv.token_logprobs_backward(x, t, w[4], g) for (x, t), w, g in zip(cases, want, d)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        k = (i + i // 4) % 4
        with torch.cuda.stream(streams[i % 2]):
            out = nv.token_logprobs(*cases[k], top=20)
            got.append((k, out, nv.token_logprobs_backward(*cases[k], out[4], d[k])))
    torch.cuda.synchronize()
    for k, out, grad in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want[k])) and torch.equal(grad, grads[k])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab,top", [(513, 328320, 0), (513, 328321, 20), (600, 400000, 64), (600, 400000, 0)])
def test_many_long_rows(nv, rows, vocab, top, dtype):
    """More rows than are shared among workgroups, of lengths at which fewer would be: the first, the middle and the
    last one against 64 bits, all of them with the bits of calls for fewer rows that are a workgroup's each."""
    x = torch.randn(rows, vocab, generator=torch.Generator("cuda").manual_seed(1), device="cuda").mul_(2.5).to(dtype)
    tokens = tokens_of(rows, 2, vocab, 3, 0.2)
    at = [0, rows // 2, rows - 1]
    tokens[at, 0] = tokens[at, 0].clamp(min=0)
    assert nv.lib().nvfp4_token_logprobs_workspace(rows, vocab, top) == 0
    got = nv.token_logprobs(x, tokens.cuda(), top=top)
    r = reference(x[at], tokens[at], 1.0, top)
    bound = lambda v: r["dz"][:, None] + U * (8 * v.abs() + 4 * r["z"][:, None])
    logp, entropy, top_logp, top_index, stats = [None if v is None else v.cpu()[at] for v in got]
    near(logp, r["logp"], bound(r["logp"]))
    near(entropy, r["h"], r["dh"])
    near(stats[:, 1], r["z"], r["dz"] + 2 * U * r["z"])
    assert torch.equal(stats[:, 0].double(), r["m"])
    if top:
        assert torch.equal(top_index, r["top"])
        near(top_logp, r["top_logp"], bound(r["top_logp"]))
    for part in (slice(0, 300), slice(rows - 300, rows)):
        for a, b in zip(got, nv.token_logprobs(x[part], tokens[part].cuda(), top=top)):
            assert (a is None and b is None) or torch.equal(a[part], b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [2, 2100])
@pytest.mark.parametrize("top", [1, 2, 5, 20, 24, 64])
def test_fewer_entries_than_alternatives(nv, rows, top, dtype):
    """Rows of every length up to about twice `top` vectors of 16 bytes with one entry above -inf, with two in one
    vector, with top - 1 and with `top` of them: the others follow in their order."""
    n = 16 // dtype.itemsize
    for vocab in [v for vectors in range(1, 2 * top + 10) for v in (vectors * n - 1, vectors * n) if v >= top]:
        for live in {1, min(2, vocab), top, max(top - 1, 1)}:
            row = torch.full((vocab,), -INF)
            at = torch.arange(live) + vocab // 2 if live <= 2 else torch.randperm(vocab, generator=gen(vocab))[:live]
            row[at % vocab] = torch.randn(live, generator=gen(live)).to(dtype).float()
            want = torch.sort(row, descending=True, stable=True)
            index = torch.full((rows, top), -5, device="cuda")
            logp = torch.full((rows, top), 5.0, device="cuda")
            x = row.to(dtype).cuda().expand(rows, vocab).contiguous()
            nv.token_logprobs(x, top=top, top_logp=logp, top_index=index)
            assert torch.equal(index.cpu(), want.indices[:top].expand(rows, top)), (vocab, live)
            few = torch.log_softmax(row.double(), 0)[want.indices[:top]]
            # (a dozen roundings of numbers below 16, and up to 64 terms)
            assert torch.equal(torch.isinf(logp[0].cpu()), torch.isinf(few))
            assert (logp.cpu() - few).nan_to_num(0.0, 0.0, 0.0).abs().max() <= 16 * 16 * U + 64 * U


@pytest.mark.parametrize("kind", ["model", "masked", "lowest", "equal", "ties"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("T", [1e-37, 1e-36, 1e-20, 1e-3, 1e5, 1e30])
def test_backward_at_extreme_temperatures(nv, T, entropy, dtype, kind):
    """Entries of probability 0 have a gradient of 0 however large 1 / T is."""
    x = logits_of((3, 500), 5, kind).to(dtype).cuda()
    tokens = tokens_of(3, 4, 500, 3)
    tokens[0, 0] = x[0].argmax().item()
    check_backward(nv, x, tokens, torch.tensor(T, dtype=F32).item(), 2, entropy)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [50001, 131072])
def test_in_place_strides_and_guards_of_shared_rows(nv, vocab, dtype):
    """The same of rows that several workgroups share, with a workspace between guards."""
    assert nv.lib().nvfp4_token_logprobs_workspace(5, vocab, 9) > 0
    test_in_place_strides_and_guards(nv, vocab, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab,top", [(5, 50001, 64), (1, 40960, 64), (64, 41000, 1), (2, 300003, 64), (3, 90000, 0)])
def test_shared_rows_between_guards(nv, rows, vocab, top, dtype):
    """Every output and the workspace of rows that several workgroups share, whatever they held before."""
    need = nv.lib().nvfp4_token_logprobs_workspace(rows, vocab, top)
    assert need > 0
    x, tokens = logits_of((rows, vocab), 7).to(dtype).cuda(), tokens_of(rows, 3, vocab, 1, 0.2).cuda()
    tokens[-1] = -1 if rows > 1 else 5
    want = nv.token_logprobs(x, tokens, top=top)
    for byte in (0, 0x7F, 0xFF):
        held = [torch.full((size + 64,), byte, dtype=torch.uint8, device="cuda")
                for size in (rows * 12, rows * 4, rows * top * 4, rows * top * 8, rows * 8, need)]
        mid = [t[32:-32] for t in held]
        logp, entropy, top_logp, stats = (mid[i].view(torch.float32) for i in (0, 1, 2, 4))
        nv.token_logprobs(x, tokens, top=top, logp=logp.view(rows, 3), entropy=entropy, stats=stats.view(rows, 2),
                          top_logp=top_logp.view(rows, top) if top else None,
                          top_index=mid[3].view(torch.int64).view(rows, top) if top else None, workspace=mid[5])
        for t in held:
            assert (t[:32] == byte).all() and (t[-32:] == byte).all()
        for w, t in zip(want, mid):
            assert w is None or torch.equal(w.view(-1).view(torch.uint8), t)


@pytest.mark.parametrize("vocab", [60000, 140001])
def test_tokens_that_are_none_or_beyond_of_shared_rows(nv, vocab):
    assert nv.lib().nvfp4_token_logprobs_workspace(4, vocab, 3) > 0
    test_tokens_that_are_none_or_beyond(nv, 4, vocab)
