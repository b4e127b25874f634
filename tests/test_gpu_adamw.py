"""The AdamW step on the GPU: against the update in 64 bits, and bit for bit against its steps in
binary32 (numpy rounds each operation once, as the kernel does).

Tolerances against 64 bits, u = 2^-24: m and v take three roundings of their terms and the
coefficients' own; sqrt, product, sum, quotient, product and difference add one each, so the
update is off by at most 16 u of itself plus its inputs' error, and p by 4 u of itself.
"""
from __future__ import annotations

import math
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
BLOCK = 128
ARGS = dict(lr=3e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)


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


def place(values, dtype, skew):
    """`values` in memory that starts `skew` elements into an allocation, canaries around."""
    n = values.numel()
    buf = torch.zeros(n + skew + 16, device="cuda", dtype=torch.uint8 if dtype == E8 else dtype)
    buf = buf.view(dtype) if dtype == E8 else buf
    view = buf[skew:skew + n]
    view.copy_(values.to(dtype))
    return view


def make(sizes, ptype, gtype, master, eight, skew=0, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed + sum(sizes))
    r = lambda n: torch.randn(n, generator=gen, device="cuda")
    params, grads, copies, avg, sq, avg_s, sq_s = [], [], [], [], [], [], []
    for k, n in enumerate(sizes):
        p = 0.05 * r(n)
        size = torch.exp(r(n) - k % 5)
        m, v = 0.3 * size * r(n), (size * (0.5 + torch.rand(n, generator=gen, device="cuda"))).square()
        params.append(place(p, ptype, skew))
        grads.append(place(size * r(n), gtype, skew))
        copies.append(place(params[-1].float() + 1e-5 * r(n), F, skew))
        if eight:
            for x, codes, scales in ((m, avg, avg_s), (v.sqrt(), sq, sq_s)):
                x = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
                s = x.abs().amax(1) / 448
                codes.append(place((x / s[:, None].clamp(min=1e-30)).clamp(-448, 448).reshape(-1)[:n], E8, skew))
                scales.append(s)
        else:
            avg.append(place(m, F, skew))
            sq.append(place(v, F, skew))
    return dict(params=params, grads=grads, master=copies if master else None, avg=avg, sq=sq,
                avg_s=avg_s if eight else None, sq_s=sq_s if eight else None)


def copy(s):
    return {k: None if v is None else [t.clone() for t in v] for k, v in s.items()}


def step(nv, s, **kw):
    plan = nv.adamw_plan(s["params"], s["avg"], s["sq"], master=s["master"], avg_scale=s["avg_s"],
                         sq_scale=s["sq_s"])
    nv.adamw_step(plan, s["grads"], **{**ARGS, **kw})


def f64(t, scale=None):
    x = t.float().double() if t.dtype == E8 else t.double()
    return x if scale is None else x * scale.double().repeat_interleave(BLOCK)[:x.numel()]


def reference(s, k, t, scale=None):
    """The update of tensor k in 64 bits -> p, m, v and the tolerances of p, m, v."""
    lr, (b1, b2), eps, wd = ARGS["lr"], ARGS["betas"], ARGS["eps"], ARGS["weight_decay"]
    g = s["grads"][k].double() * (1.0 if scale is None else float(scale))
    m = f64(s["avg"][k], s["avg_s"][k] if s["avg_s"] else None)
    v = f64(s["sq"][k], s["sq_s"][k] if s["sq_s"] else None)
    if s["sq_s"]:
        v = v * v
    p = (s["master"] or s["params"])[k].double()
    size = b1 * m.abs() + (1 - b1) * g.abs()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    tm, tv = 6 * U * size, 8 * U * v
    down = (v / (1 - b2 ** t)).sqrt() + eps
    rate = lr / (1 - b1 ** t)
    upd = rate * m / down
    want = p * (1 - lr * wd) - upd
    tp = 3 * U * p.abs() + 2 * U * want.abs() + 16 * U * upd.abs() + rate * tm / down
    return want, m, v, tp, tm + 1e-40, tv + 1e-40


def inside(got, want, tol, what):
    off = (got.double() - want).abs()
    assert (off <= tol).all(), "%s: %.3g times the tolerance" % (what, float((off / tol).max()))


SIZES = [1, 7, 8, 9, 0, 127, 128, 129, 1000, 8191, 8192, 8193, 0, 16384, 100003, 3]
KINDS = [(F, False), (BF, True), (BF, False)]


def check(nv, s, t, seed=5, scale=None, amax=False, old=None):
    old = old or copy(s)
    n = len(s["params"])
    top = torch.full((n,), -1.0, device="cuda") if amax else None
    c = None if scale is None else torch.full((1,), scale, device="cuda")
    step(nv, s, step=t, seed=seed, grad_scale=c, amax=top)
    for k in range(n):
        p, m, v, tp, tm, tv = reference(old, k, t, None if scale is None else c.item())
        if p.numel() == 0:
            assert top is None or top[k].item() == 0
            continue
        param, alone = s["params"][k], s["params"][k].dtype == BF and s["master"] is None
        if s["master"]:
            inside(s["master"][k], p, tp, "master")
            assert torch.equal(param, s["master"][k].to(BF))
        elif alone:                  # one of the two bf16 neighbours: within one step of it
            inside(param, p, tp + 2.0 ** -7 * p.abs() + 2.0 ** -133, "bf16 parameter")
        else:
            inside(param, p, tp, "parameter")
        if s["avg_s"]:
            low = v.sqrt()
            for name, x, tol, codes, scales in (("m", m, tm, s["avg"], s["avg_s"]),
                                                ("sqrt v", low, 8 * U * low, s["sq"], s["sq_s"])):
                rows = torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)
                want = rows.abs().amax(1) / 448
                near = torch.nn.functional.pad(tol, (0, -x.numel() % BLOCK)).view(-1, BLOCK).amax(1) / 448
                inside(scales[k], want, near + 2 * U * want, name + " scale")
                y = x / scales[k].double().clamp(min=1e-300).repeat_interleave(BLOCK)[:x.numel()]
                got = codes[k].float().double()
                # a step of the grid at |y|: 2^(floor(log2 |y|) - 3), 2^-9 below 2^-6
                grid = 2.0 ** (torch.floor(torch.log2((y.abs() * (1 + 1e-5)).clamp(min=2.0 ** -6))) - 3)
                inside(got, y, grid * (1 + 1e-4) + 1e-5 * y.abs(), name + " codes")
                if name != "m":
                    assert ((got > 0) == (x > 0)).all()
        else:
            inside(s["avg"][k], m, tm, "m")
            inside(s["sq"][k], v, tv, "v")
        if amax:
            assert top[k].item() == param.float().abs().max().item()


@pytest.mark.parametrize("eight", [False, True], ids=["f32", "e4m3"])
@pytest.mark.parametrize("gtype", [BF, F], ids=str)
@pytest.mark.parametrize("ptype,master", KINDS, ids=["f32", "master", "bf16"])
def test_step(nv, ptype, master, gtype, eight):
    for skew in (0, 1, 3):
        say("[adamw]", ptype, master, gtype, eight, skew)
        s = make(SIZES, ptype, gtype, master, eight, skew)
        for t in (1, 2, 3):                       # the second step runs on the first one's states
            check(nv, s, t, amax=t != 2, scale=0.37 if t == 3 else None)


def test_more_tensors_than_a_launch_takes(nv):
    sizes = [1 + (37 * k) % 5000 for k in range(131)]
    for ptype, master, eight in ((F, False, False), (BF, False, True)):
        check(nv, make(sizes, ptype, F, master, eight), 1, amax=True)
    check(nv, make([0, 0, 5, 0], F, F, False, False), 1, amax=True)
    check(nv, make([0] * 60 + [9], BF, BF, True, True), 1, amax=True)
    check(nv, make([0] * 3, F, F, False, False), 1, amax=True)


# ------------------------------------------------------------------ binary32, bit for bit
def mix(h):
    h = np.uint32(h) if np.isscalar(h) else h
    with np.errstate(over="ignore"):
        h = h ^ (h >> np.uint32(16))
        h = (h * np.uint32(0x7FEB352D)).astype(np.uint32)
        h = h ^ (h >> np.uint32(15))
        h = (h * np.uint32(0x846CA68B)).astype(np.uint32)
        return h ^ (h >> np.uint32(16))


def e4m3_cut(y, bits):
    """y >= 0 to E4M3 by adding the bits below the kept ones: in steps of the format's grid."""
    y = y.astype(np.float32)
    e = np.maximum(np.floor(np.log2(np.maximum(y, np.float32(2.0 ** -30)))), -6)
    out = np.empty_like(y)
    low = y < 2.0 ** -6
    moved = np.where(low, y + np.float32(2.0 ** -6), y).astype(np.float32)
    word = moved.view(np.uint32).astype(np.uint64) + bits.astype(np.uint64)
    cut = ((word >> np.uint64(20)) << np.uint64(20)).astype(np.uint32).view(np.float32)
    out = np.where(low, cut - np.float32(2.0 ** -6), cut)
    assert (np.abs(out - y) <= 2.0 ** (e - 3)).all()
    return np.minimum(out, np.float32(448))


@pytest.mark.parametrize("ptype,master", KINDS, ids=["f32", "master", "bf16"])
@pytest.mark.parametrize("eight", [False, True], ids=["f32", "e4m3"])
def test_bits(nv, ptype, master, eight):
    t, seed, f = 7, 0xDEADBEEF, np.float32
    lr, (b1, b2), eps, wd = ARGS["lr"], ARGS["betas"], ARGS["eps"], ARGS["weight_decay"]
    s = make([1000, 129, 20001], ptype, BF, master, eight)
    old = copy(s)
    step(nv, s, step=t, seed=seed)
    key = mix(mix(np.uint32(seed)) ^ np.uint32(t))
    host = lambda x: x.float().cpu().numpy()
    for k in range(3):
        g, m, v = host(old["grads"][k]), host(old["avg"][k]), host(old["sq"][k])
        n = g.size
        if eight:
            m = m * np.repeat(host(old["avg_s"][k]), BLOCK)[:n]
            v = v * np.repeat(host(old["sq_s"][k]), BLOCK)[:n]
            v = v * v
        m = m * f(b1) + g * f(1 - b1)
        v = v * f(b2) + (g * g) * f(1 - b2)
        low = np.sqrt(v)
        p = host((old["master"] or old["params"])[k])
        p = p * f(1 - lr * wd) - (m / (low * f(1 / math.sqrt(1 - b2 ** t)) + f(eps))) * f(lr / (1 - b1 ** t))
        with np.errstate(over="ignore"):
            bits = mix(np.arange(n, dtype=np.uint32) + mix(key ^ np.uint32(k)))
        if eight:
            for x, r, codes, scales, positive in ((m, bits & np.uint32(0xFFFFF), s["avg"], s["avg_s"], False),
                                                  (low, bits >> np.uint32(12), s["sq"], s["sq_s"], True)):
                rows = np.pad(x, (0, -n % BLOCK)).reshape(-1, BLOCK)
                scale = np.abs(rows).max(1) * f(1 / 448)
                assert np.array_equal(host(scales[k]).view(np.uint32), scale.view(np.uint32))
                y = x * np.repeat(f(1) / scale, BLOCK)[:n]
                want = np.copysign(e4m3_cut(np.abs(y), r), y)
                if positive:
                    want = np.where(x > 0, np.maximum(want, f(2.0 ** -9)), want)
                assert np.array_equal(host(codes[k]), want)
        else:
            assert np.array_equal(host(s["avg"][k]).view(np.uint32), m.view(np.uint32))
            assert np.array_equal(host(s["sq"][k]).view(np.uint32), v.view(np.uint32))
        # the quotient may be off by two steps: by 2^-22 of the update
        off = 2.0 ** -22 * np.abs(p - host((old["master"] or old["params"])[k])) + 2.0 ** -23 * np.abs(p)
        if ptype == BF and not master:
            with np.errstate(over="ignore"):
                r = ((bits * np.uint32(0x9E3779B1)).astype(np.uint32) >> np.uint32(16)).astype(np.uint64)
            word = (p.view(np.uint32) & np.uint32(0x7FFFFFFF)).astype(np.uint64) + r
            want = np.copysign((word >> np.uint64(16) << np.uint64(16)).astype(np.uint32).view(np.float32), p)
            differ = np.mean(host(s["params"][k]) != want)
            assert differ <= 2e-3, differ       # a step of p moves the cut in 2 of 2^16 elements or so
        else:
            got = host((s["master"] or s["params"])[k])
            assert (np.abs(got.astype(np.float64) - p) <= off).all()


def test_stochastic_rounding_is_unbiased(nv):
    """A bf16 parameter that moves by a hundredth of its step per call gets there on average, and
    so does an 8-bit second moment that moves by a tenth of a step: both stand still under
    round-to-nearest.  200,000 elements; the mean of n independent roundings is within 6 sigma."""
    n = 200_000
    p = torch.full((n,), 1.0, device="cuda", dtype=BF)
    g = torch.full((n,), 1.0, device="cuda")
    plan = nv.adamw_plan([p])
    steps, lr = 20, 2.0 ** -7 / 100
    for t in range(1, steps + 1):
        nv.adamw_step(plan, [g], step=t, lr=lr, betas=(0.0, 0.0), eps=0.0, weight_decay=0.0, seed=11)
    moved = (1.0 - p.double()).mean().item()
    sigma = 2.0 ** -7 * math.sqrt(0.01 * steps / n)
    assert abs(moved - steps * lr) <= 6 * sigma + 1e-6, (moved, steps * lr)
    assert len(p.unique()) > 1

    # sqrt(v) from 100 towards 90 (beta2 = 0.99: v moves by 0.2 % a step, a code's step is 1/16);
    # one element per block holds the scale at 448
    v0, g0 = 100.0, 90.0
    blocks = n // BLOCK
    codes = torch.full((blocks, BLOCK), v0, device="cuda")
    codes[:, 0] = 448.0
    grad = torch.full((blocks, BLOCK), g0, device="cuda")
    grad[:, 0] = 448.0
    codes = codes.view(-1).to(E8)
    start = codes.float().view(blocks, BLOCK)[0, 1].item()          # 96 or 104: the grid
    zero = torch.zeros(blocks * BLOCK, device="cuda")
    plan = nv.adamw_plan([zero], [torch.zeros_like(zero).to(E8)], [codes],
                         avg_scale=[torch.zeros(blocks, device="cuda")],
                         sq_scale=[torch.ones(blocks, device="cuda")])
    for t in range(1, 31):
        nv.adamw_step(plan, [grad.view(-1)], step=t, lr=0.0, betas=(0.9, 0.99), seed=3)
    got = codes.float().view(blocks, BLOCK)[:, 1:].double() * plan.sq_scale[0].double()[:, None]
    want = math.sqrt(g0 ** 2 + (start ** 2 - g0 ** 2) * 0.99 ** 30)
    # the mean of sqrt(v) follows v's mean up to the roundings' spread: steps of 8 around 96
    spread = got.std().item()
    assert abs(got.mean().item() - want) <= 6 * spread / math.sqrt(got.numel()) + spread ** 2 / want
    assert spread > 0


def test_bits_depend_on_seed_step_tensor_and_place_only(nv):
    sizes = [5000, 5000]
    def run(seed, t, extra=False):
        s = make(sizes, BF, F, False, True, seed=1)
        s["params"][1].copy_(s["params"][0])
        s["grads"][1].copy_(s["grads"][0])
        for k in ("avg", "sq", "avg_s", "sq_s"):
            s[k][1].copy_(s[k][0])
        step(nv, s, step=t, seed=seed)
        return s["params"]
    a, b, c = run(1, 5), run(1, 5), run(2, 5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert not torch.equal(a[0], a[1]) and not torch.equal(a[0], c[0])
    # a step of zero rate and decay leaves a representable parameter alone
    s = make([3000], BF, F, False, True)
    old = copy(s)
    plan = nv.adamw_plan(s["params"], s["avg"], s["sq"], avg_scale=s["avg_s"], sq_scale=s["sq_s"])
    nv.adamw_step(plan, s["grads"], step=1, lr=0.0)
    assert torch.equal(s["params"][0], old["params"][0])


@pytest.mark.parametrize("eight", [False, True], ids=["f32", "e4m3"])
def test_non_finite_gradients_stay_in_their_place(nv, eight):
    for bad in (float("nan"), float("inf"), 1e30):
        for ptype, master in KINDS:
            s = make([1000, 300], ptype, F, master, eight)
            clean = copy(s)
            s["grads"][0][200] = bad
            step(nv, s, step=3)
            step(nv, clean, step=3)
            p = s["params"][0]
            if bad != 1e30:
                assert torch.isnan(p[200])
            keep = torch.ones(1000, dtype=torch.bool, device="cuda")
            keep[200] = False
            assert torch.equal(p[keep], clean["params"][0][keep])
            assert torch.equal(s["params"][1], clean["params"][1])
            if eight:        # the block of element 200 reads back as not finite; the others do not
                back = f64(s["avg"][0], s["avg_s"][0])
                second = f64(s["sq"][0], s["sq_s"][0])
                if bad != 1e30:
                    assert not torch.isfinite(back[200]) and not torch.isfinite(back[128:256]).any()
                assert not torch.isfinite(second[128:256]).any()
                assert torch.isfinite(back[:128]).all() and torch.isfinite(second[256:]).all()
            elif bad != 1e30:
                assert torch.isnan(s["avg"][0][200]) or torch.isinf(s["avg"][0][200])


def test_zero_states_and_zero_gradients(nv):
    for eight in ("f32", "e4m3"):
        for ptype, master in KINDS:
            p = torch.linspace(-1, 1, 500, device="cuda").to(ptype)
            want = p.clone()
            plan = nv.adamw_plan([p], state=eight, master=True if master else None)
            nv.adamw_step(plan, [torch.zeros(500, device="cuda")], step=1, lr=0.1, weight_decay=0.0)
            assert torch.equal(p, want)                   # 0 / (0 + eps) = 0
            assert (plan.exp_avg[0].float() == 0).all() and (plan.exp_avg_sq[0].float() == 0).all()
            # the first real step moves every parameter by lr against its gradient's sign
            g = torch.where(torch.arange(500, device="cuda") % 2 == 0, 1e-3, -2e-3)
            nv.adamw_step(plan, [g], step=1, lr=0.125, eps=0.0, weight_decay=0.0)
            got = (plan.master[0] if master else p).float() - want.float()
            tol = 2.0 ** -7 if ptype == BF and not master else 1e-6
            assert ((got + 0.125 * g.sign()).abs() <= tol).all()


def test_amax_serves_the_quantization(nv):
    gen = torch.Generator("cuda").manual_seed(1)
    params = [torch.randn(64, 256, generator=gen, device="cuda").to(BF) for _ in range(3)]
    grads = [torch.randn(64, 256, generator=gen, device="cuda").to(BF) for _ in range(3)]
    for state in ("f32", "e4m3"):
        for master in (None, True):
            plan = nv.adamw_plan(params, master=master, state=state)
            amax = torch.empty(3, device="cuda")
            nv.adamw_step(plan, grads, step=1, lr=0.01, amax=amax)
            for k, p in enumerate(params):
                assert torch.equal(amax[k:k + 1], nv.amax(p))
                a, b = nv.quantize(p), nv.quantize_from_amax(p, amax[k:k + 1])
                assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_graph_replays_and_streams(nv):
    s = make([5000, 70000, 3], BF, BF, False, True)
    old, c, amax = copy(s), torch.full((1,), 0.5, device="cuda"), torch.zeros(3, device="cuda")
    plan = nv.adamw_plan(s["params"], s["avg"], s["sq"], avg_scale=s["avg_s"], sq_scale=s["sq_s"])
    state = s["params"] + s["avg"] + s["sq"] + s["avg_s"] + s["sq_s"]
    start = old["params"] + old["avg"] + old["sq"] + old["avg_s"] + old["sq_s"]
    raw = lambda t: t.view(torch.uint8) if t.dtype == E8 else t

    def reset():
        for t, o in zip(state, start):
            raw(t).copy_(raw(o))
        amax.fill_(7)
    work = lambda: nv.adamw_step(plan, s["grads"], step=2, lr=1e-2, grad_scale=c, amax=amax, seed=4)
    work()
    torch.cuda.synchronize()
    want = [raw(t).clone() for t in state] + [amax.clone()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for turn in range(4):
        reset()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(raw(t), w) for t, w in zip(state + [amax], want)), turn
    reset()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    assert all(torch.equal(raw(t), w) for t, w in zip(state + [amax], want))


def test_nothing_beyond_the_tensors_is_written(nv):
    for eight in (False, True):
        for ptype, master in KINDS:
            gen = torch.Generator("cuda").manual_seed(2)
            sizes, guard = [1, 130, 4097], 64
            kinds = {"params": ptype, "avg": E8 if eight else F, "sq": E8 if eight else F}
            if master:
                kinds["master"] = F
            if eight:
                kinds.update(avg_s=F, sq_s=F)
            bufs, views = {}, {}
            for name, dtype in kinds.items():
                bufs[name], views[name] = [], []
                for n in sizes:
                    n = -(-n // BLOCK) if name.endswith("_s") else n
                    b = torch.full((n + 2 * guard,), 1.5, device="cuda").to(dtype)
                    v = b[guard:guard + n]
                    v.copy_((torch.rand(n, generator=gen, device="cuda") + 0.1).to(dtype))
                    bufs[name].append(b)
                    views[name].append(v)
            grads = [torch.randn(n, generator=gen, device="cuda") for n in sizes]
            plan = nv.adamw_plan(views["params"], views["avg"], views["sq"], master=views.get("master"),
                                 avg_scale=views.get("avg_s"), sq_scale=views.get("sq_s"))
            nv.adamw_step(plan, grads, step=1, lr=0.1)
            for name, bs in bufs.items():
                for b in bs:
                    x = b.float()
                    assert (x[:guard] == 1.5).all() and (x[-guard:] == 1.5).all(), name


def test_refusals(nv):
    p, g = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    plan = nv.adamw_plan([p])
    ok = dict(step=1, lr=0.1)
    for err, call in (
            (TypeError, lambda: nv.adamw_plan([p.half()])),
            (ValueError, lambda: nv.adamw_plan([p], state="e5m2")),
            (ValueError, lambda: nv.adamw_plan([p], [p])),
            (ValueError, lambda: nv.adamw_plan([p], avg_scale=[p])),
            (ValueError, lambda: nv.adamw_plan([p], master=True)),
            (TypeError, lambda: nv.adamw_plan([p, p.to(BF)])),
            (TypeError, lambda: nv.adamw_plan([p], [p.to(BF)], [p.to(BF)])),
            (ValueError, lambda: nv.adamw_plan([p], [p.to(E8)], [p.to(E8)])),
            (ValueError, lambda: nv.adamw_plan([p], [p[:3]], [p])),
            (ValueError, lambda: nv.adamw_plan([p], [p.clone()], [p.clone(), p.clone()])),
            (ValueError, lambda: nv.adamw_plan([torch.zeros(8, 8, device="cuda").t()[:, :4]])),
            (ValueError, lambda: nv.adamw_step(plan, [], **ok)),
            (ValueError, lambda: nv.adamw_step(plan, [g[:5]], **ok)),
            (ValueError, lambda: nv.adamw_step(plan, [g.cpu()], **ok)),
            (TypeError, lambda: nv.adamw_step(plan, [g.half()], **ok)),
            (ValueError, lambda: nv.adamw_step(plan, [g], seed=-1, **ok)),
            (ValueError, lambda: nv.adamw_step(plan, [g], amax=g, **ok)),
            (TypeError, lambda: nv.adamw_step(plan, [g], grad_scale=g[:1].double(), **ok)),
            (nv.NVFP4Error, lambda: nv.adamw_step(plan, [g], step=0, lr=0.1)),
            (nv.NVFP4Error, lambda: nv.adamw_step(plan, [g], betas=(1.0, 0.9), **ok)),
            (nv.NVFP4Error, lambda: nv.adamw_step(plan, [p], **ok))):
        with pytest.raises(err):
            call()


def test_parameters_that_moved(nv):
    """New memory of the same size is taken; of another size, type or number it is refused."""
    params = [torch.nn.Parameter(torch.ones(n, device="cuda")) for n in (300, 40)]
    plan = nv.adamw_plan(params)
    grads = [torch.ones_like(p) for p in params]
    old = params[0].data
    params[0].data = torch.full((300,), 5.0, device="cuda")
    nv.adamw_step(plan, grads, step=1, lr=0.5, weight_decay=0.0)
    assert (old == 1).all() and ((params[0] - 4.5).abs() < 1e-5).all() and ((params[1] - 0.5).abs() < 1e-5).all()
    params[1].data = torch.ones(39, device="cuda")
    for _ in range(2):
        with pytest.raises(ValueError, match="params"):
            nv.adamw_step(plan, grads, step=2, lr=0.5)
    params[1].data = torch.ones(40, device="cuda")
    plan.exp_avg[0] = torch.zeros(300, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="exp_avg"):
        nv.adamw_step(plan, grads, step=2, lr=0.5)
    plan.exp_avg[0] = torch.zeros(300, device="cuda")
    plan.exp_avg.pop()
    with pytest.raises(ValueError, match="exp_avg"):
        nv.adamw_step(plan, grads, step=2, lr=0.5)
    assert ((params[0] - 4.5).abs() < 1e-5).all() and (params[1] == 1).all()


def test_a_tensor_past_32_bits(nv):
    """Elements past 2^32 are updated as they would be by themselves; the random bits do not repeat
    there."""
    n, size = (1 << 32) + 5000, 5000
    gen = torch.Generator("cuda").manual_seed(6)
    places = (0, (1 << 31) - 77, (1 << 32) - 2048, n - size)
    grad = torch.randn(size, generator=gen, device="cuda").to(BF)
    g = torch.zeros(n, device="cuda", dtype=BF)
    for at in places:
        g[at:at + size] = grad
    args = dict(step=3, lr=0.01, weight_decay=0.0)
    p = torch.ones(n, device="cuda")
    plan = nv.adamw_plan([p])
    nv.adamw_step(plan, [g], **args)
    few = torch.ones(size, device="cuda")
    want = nv.adamw_plan([few])
    nv.adamw_step(want, [grad], **args)
    # the last place begins within the one before it, which ends there
    first = {at: min([b - at for b in places if b > at] + [size]) for at in places}
    for at, m in first.items():
        assert torch.equal(p[at:at + m], few[:m]) and torch.equal(plan.exp_avg[0][at:at + m], want.exp_avg[0][:m])
    assert (p[size:1 << 20] == 1).all() and (p[1 << 31:][size:1 << 20] == 1).all()
    del p, plan
    torch.cuda.empty_cache()
    p = torch.ones(n, device="cuda", dtype=BF)
    plan = nv.adamw_plan([p], state="e4m3")
    nv.adamw_step(plan, [g], **args)
    for at, m in first.items():
        got, exact = p[at:at + m].float(), few[:m]
        assert ((got - exact).abs() <= 2.0 ** -7).all() and (got != 1).any()
    tail = p[n - size:]
    alone = torch.ones(size, device="cuda", dtype=BF)
    nv.adamw_step(nv.adamw_plan([alone], state="e4m3"), [grad], **args)
    assert not torch.equal(tail, alone) and not torch.equal(p[:size], tail)
    assert torch.equal(p[:first[0]], alone[:first[0]])


def test_parameters_that_changed_where_they_are(nv):
    """A view of a tensor at its own address, of another size, order or type, is refused for every kind
    of tensor, as are such gradients; the step leaves everything as it was."""
    for ptype, state, master in ((F, "f32", None), (BF, "f32", True), (BF, "e4m3", None)):
        params = [torch.nn.Parameter(torch.ones(40, 40, device="cuda", dtype=ptype)) for _ in range(3)]
        plan = nv.adamw_plan(params, state=state, master=master)
        grads = [torch.ones(40, 40, device="cuda") for _ in params]
        nv.adamw_step(plan, grads, step=1, lr=0.5)
        lists = {k: getattr(plan, k) for k in plan.KINDS if getattr(plan, k) is not None}
        was = [t.detach().clone() for v in lists.values() for t in v]
        for kind, tensors in {**lists, "grads": grads}.items():
            whole = tensors[1].data
            others = [(whole[:2] if whole.dim() > 1 else whole[:5], ValueError)]
            if whole.dim() > 1:
                others.append((whole.t(), ValueError))
            half = whole.view(torch.float16 if whole.dtype != E8 else torch.uint8).flatten()[:whole.numel()]
            others.append((half.view(whole.shape), TypeError))
            for other, error in others:
                assert other.data_ptr() == whole.data_ptr()
                if kind == "params" and other.dtype == whole.dtype:
                    tensors[1].data = other
                else:
                    keep = tensors[1]
                    tensors[1] = other
                for _ in range(2):
                    with pytest.raises(error, match=kind):
                        nv.adamw_step(plan, grads, step=2, lr=0.5)
                if kind == "params" and other.dtype == whole.dtype:
                    tensors[1].data = whole
                else:
                    tensors[1] = keep
        torch.cuda.synchronize()
        assert all(torch.equal(t.view(torch.uint8), w.view(torch.uint8))
                   for t, w in zip((t.detach() for v in lists.values() for t in v), was))
        # what is alike but elsewhere, or of another shape, is taken
        params[1].data = params[1].data.clone().view(1600)
        params[2].data = params[2].data.view(20, 80)
        nv.adamw_step(plan, grads, step=2, lr=0.5)
        assert torch.equal(params[0].view(-1), params[1]) and torch.equal(params[0].view(-1), params[2].view(-1)) \
            or (ptype == BF and master is None)


@pytest.mark.parametrize("eps", [0.0, 1e-8])
@pytest.mark.parametrize("ptype,master", KINDS, ids=["f32", "master", "bf16"])
def test_second_moments_below_the_normal_numbers(nv, ptype, master, eps):
    """8-bit states, gradients whose squares are subnormal: blocks of such gradients alone, and beside
    ordinary ones, and beside one whose square is infinite (its block reads back as not finite).  sqrt(v),
    the scales and the codes bit for bit as numpy has them, no code of a v > 0 is 0, and the update is
    the one of binary32 (tolerance as in test_bits)."""
    t, seed, f = 1, 77, np.float32
    lr, (b1, b2), wd = ARGS["lr"], ARGS["betas"], ARGS["weight_decay"]
    gen = torch.Generator("cuda").manual_seed(12)
    sizes = (1e-18, 3e-20, 5e-21)
    grads = []
    for alone in sizes:                    # a tensor for each size: alone, beside 1, beside 4e20, a cut block
        r = torch.randn(4 * BLOCK + 37, generator=gen, device="cuda", dtype=torch.float64)
        g = alone * r.sign() * (1 + r.abs())
        g[BLOCK + 5], g[2 * BLOCK + 9], g[4 * BLOCK:4 * BLOCK + 3] = 1.0, 4e20, 0.0
        grads.append(g.float())
    params = [(0.05 * torch.randn(g.numel(), generator=gen, device="cuda")).to(ptype) for g in grads]
    old = [p.clone() for p in params]
    plan = nv.adamw_plan(params, state="e4m3", master=True if master else None)
    nv.adamw_step(plan, grads, step=t, seed=seed, eps=eps, lr=lr, betas=(b1, b2), weight_decay=wd)
    key = mix(mix(np.uint32(seed)) ^ np.uint32(t))
    host = lambda x: x.float().cpu().numpy()
    for k, g in enumerate(map(host, grads)):
        n = g.size
        with np.errstate(over="ignore"):
            m, v = g * f(1 - b1), (g * g) * f(1 - b2)
        low = np.sqrt(v)
        assert ((v > 0) == (g != 0)).all() and (v[v > 0].min() < 2.0 ** -126)
        p0 = host(old[k])
        with np.errstate(invalid="ignore", divide="ignore"):
            p = p0 * f(1 - lr * wd) - (m / (low * f(1 / math.sqrt(1 - b2 ** t)) + f(eps))) * f(lr / (1 - b1 ** t))
        with np.errstate(over="ignore"):
            bits = mix(np.arange(n, dtype=np.uint32) + mix(key ^ np.uint32(k)))
        for x, r, codes, scales, positive in (
                (m, bits & np.uint32(0xFFFFF), plan.exp_avg[k], plan.avg_scale[k], False),
                (low, bits >> np.uint32(12), plan.exp_avg_sq[k], plan.sq_scale[k], True)):
            finite = np.ones(n, bool)
            if positive:
                finite[2 * BLOCK:3 * BLOCK] = False
                assert not torch.isfinite(f64(codes, scales)[2 * BLOCK:3 * BLOCK]).any()
                x = np.where(finite, x, f(1))
            scale = np.abs(np.pad(x, (0, -n % BLOCK)).reshape(-1, BLOCK)).max(1) * f(1 / 448)
            held = np.append(finite[::BLOCK][:n // BLOCK], True)
            assert np.array_equal(host(scales)[held].view(np.uint32), scale[held].view(np.uint32)), (k, positive)
            y = x * np.repeat(f(1) / scale, BLOCK)[:n]
            want = np.copysign(e4m3_cut(np.abs(y), r), y)
            if positive:
                want = np.where(x > 0, np.maximum(want, f(2.0 ** -9)), want)
                assert ((host(codes) > 0) == (v > 0))[finite].all()
            assert np.array_equal(host(codes)[finite], want[finite]), (k, positive)
        got = host((plan.master or params)[k])
        live = g != 0 if eps == 0 else np.ones(n, bool)               # 0 / 0 where the gradient is 0
        off = 2.0 ** -22 * np.abs(p - p0) + 2.0 ** -23 * np.abs(p)
        if ptype == BF and not master:                               # one of the two bf16 neighbours
            off = off + 2.0 ** -7 * np.abs(p) + 2.0 ** -133
        assert (np.abs(got.astype(np.float64) - p)[live] <= off[live]).all(), k
        assert np.isnan(got[~live]).all()


def test_second_moments_beside_the_largest(nv):
    """The smallest and the largest roots of a block: codes of 2^-9 and 448, and a scale between."""
    g = torch.full((2 * BLOCK,), 1.8e19, device="cuda")
    g[1::2], g[BLOCK:] = 1.3e-21, 0.0
    g[BLOCK + 3] = 1.3e-21
    v = (g * g) * np.float32(1 - 0.999)
    assert v[1].item() == 2.0 ** -149
    for seed in range(4):
        plan = nv.adamw_plan([torch.zeros(2 * BLOCK, device="cuda")], state="e4m3")
        nv.adamw_step(plan, [g], step=1, lr=0.125, eps=0.0, weight_decay=0.0, seed=seed)
        codes = plan.exp_avg_sq[0].float()
        assert (codes[:BLOCK:2] == 448).all() and (codes[1:BLOCK:2] == 2.0 ** -9).all()
        assert codes[BLOCK + 3] == 448 and (codes[BLOCK:] > 0).sum() == 1
        assert plan.sq_scale[0][1].item() == np.float32(2.0 ** -74.5) * np.float32(1 / 448)
        # m / sqrt(v) with the root of the binary32 v: within 2 ulp of 0.1 g / sqrt(v), corrected
        live = g != 0
        p = plan.params[0][live].double()
        want = -0.125 * (g * np.float32(0.1))[live].double() / v[live].double().sqrt() * math.sqrt(1 - 0.999) / (1 - 0.9)
        assert ((p - want).abs() <= 2.0 ** -20 * want.abs()).all()
