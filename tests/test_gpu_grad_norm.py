"""The gradient norm over many tensors, its clipping coefficient and the scaled tensors (GPU).

The squares and sums are binary64: the norm is the correctly rounded one but for ties within 2^-20 of
half a step, so 1.01 half steps are allowed; products are compared bit for bit."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_block_scaled_amax_amd as m
    m.lib()
    return m


def plan_of(nv, sizes):
    return nv.adamw_plan([torch.zeros(n, dtype=BF16, device="cuda") for n in sizes], state="e4m3")


def grads_of(sizes, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(size * math.exp(k % 5 - 2) * torch.randn(n, generator=g)).to(dtype).cuda() for k, n in enumerate(sizes)]


def exact(grads, max_norm, eps):
    total = math.fsum(float(g.double().square().sum()) for g in grads)
    norm = math.sqrt(total)
    return norm, min(1.0, max_norm / (norm + eps))


def close(got, want):
    return abs(got.item() - want) <= 1.01 * 2.0 ** -24 * want + 2.0 ** -149


SIZES = {"one": [1], "few": [3, 1, 17], "empty ones": [0, 5, 0, 8192, 0], "chunks": [8191, 8192, 8193, 4096, 4097],
         "many": [1 + 37 * k % 1000 for k in range(777)], "exactly a table": [64] * 200, "one more": [64] * 201,
         "large": [3_000_001, 20_000_003, 5], "more chunks than workgroups": [40_000_001]}


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sizes", list(SIZES), ids=list(SIZES))
def test_norm_and_clip(nv, sizes, dtype):
    sizes = SIZES[sizes]
    plan, grads = plan_of(nv, sizes), grads_of(sizes, dtype, 1)
    norm, scale = nv.grad_norm(plan, grads, max_norm=0.3, eps=1e-3)
    want, by = exact(grads, 0.3, 1e-3)
    assert close(norm, want) and close(scale, by)
    alone, none = nv.grad_norm(plan, grads)
    assert none is None and torch.equal(alone, norm)
    products = [(g.float() * scale).to(dtype) for g in grads]
    before = [g.clone() for g in grads]
    out = [torch.full_like(g, 5.0) for g in grads]
    assert nv.clip_grads(plan, grads, scale, out=out)[0] is out[0]
    for o, p, g, b in zip(out, products, grads, before):
        assert torch.equal(o, p) and torch.equal(g, b)
    assert nv.clip_grads(plan, grads, scale)[0] is grads[0]
    for g, p in zip(grads, products):
        assert torch.equal(g, p)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_norm_within_bounds_changes_nothing(nv, dtype):
    sizes = [100, 9000]
    plan, grads = plan_of(nv, sizes), grads_of(sizes, dtype, 1)
    before = [g.clone() for g in grads]
    norm, scale = nv.grad_norm(plan, grads, max_norm=1e9)
    assert scale.item() == 1.0
    out = [torch.empty_like(g) for g in grads]
    nv.clip_grads(plan, grads, scale, out=out)
    nv.clip_grads(plan, grads, scale)
    for g, o, b in zip(grads, out, before):
        assert torch.equal(g, b) and torch.equal(o, b)
    assert nv.grad_norm(plan, grads, max_norm=0.0)[1].item() == 0.0
    zeros = [torch.zeros_like(g) for g in grads]
    norm, scale = nv.grad_norm(plan, zeros, max_norm=0.5)
    assert norm.item() == 0.0 and scale.item() == 1.0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-12, 1e18, 1e34])
def test_sizes_whose_squares_pass_32_bits(nv, size, dtype):
    sizes = [5000, 3]
    plan, grads = plan_of(nv, sizes), grads_of(sizes, dtype, 2, size)
    norm, scale = nv.grad_norm(plan, grads, max_norm=size)
    want, by = exact(grads, float(torch.tensor(size, dtype=torch.float64)), 1e-6)
    assert close(norm, want) and close(scale, by)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_values_that_are_not_finite(nv, dtype, value):
    sizes = [70, 100_000]
    plan, grads = plan_of(nv, sizes), grads_of(sizes, dtype, 2)
    grads[1][99_999] = value
    norm, scale = nv.grad_norm(plan, grads, max_norm=1.0)
    if math.isnan(value):
        assert math.isnan(norm.item()) and math.isnan(scale.item())
    else:
        assert norm.item() == INF and scale.item() == 0.0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_parts_of_a_buffer(nv, dtype):
    """Gradients that start at any element of one buffer; nothing between them is read or written."""
    sizes = [33, 8192, 1, 20_001]
    plan, grads = plan_of(nv, sizes), grads_of(sizes, dtype, 3)
    held = torch.full((40_000,), NAN, dtype=dtype, device="cuda")
    to = torch.full((40_000,), NAN, dtype=dtype, device="cuda")
    at, parts, outs, inside = 7, [], [], torch.zeros(40_000, dtype=torch.bool, device="cuda")
    for g in grads:
        parts.append(held[at:at + g.numel()])
        outs.append(to[at + 1:at + 1 + g.numel()])
        parts[-1].copy_(g)
        inside[at:at + g.numel()] = True
        at += g.numel() + 13
    norm, scale = nv.grad_norm(plan, parts, max_norm=0.1)
    assert close(norm, exact(grads, 0.1, 1e-6)[0])
    nv.clip_grads(plan, parts, scale, out=outs)
    nv.clip_grads(plan, parts, scale)
    for p, o, g in zip(parts, outs, grads):
        assert torch.equal(p, (g.float() * scale).to(dtype)) and torch.equal(o, p)
    assert torch.isnan(held[~inside]).all() and torch.isnan(to[1:][~inside[:-1]]).all() and torch.isnan(to[0])


def test_the_step_takes_the_coefficient(nv):
    """adamw_step(grad_scale=scale) is adamw_step on the gradients that clip_grads leaves, in 32 bits."""
    sizes = [1000, 77]
    make = lambda: nv.adamw_plan([torch.ones(n, device="cuda") for n in sizes])
    one, two, grads = make(), make(), grads_of(sizes, F32, 4)
    norm, scale = nv.grad_norm(one, grads, max_norm=0.5)
    nv.adamw_step(one, grads, step=1, lr=0.1, grad_scale=scale)
    nv.adamw_step(two, nv.clip_grads(two, grads, scale), step=1, lr=0.1)
    for a, b in zip(one.params + one.exp_avg + one.exp_avg_sq, two.params + two.exp_avg + two.exp_avg_sq):
        assert torch.equal(a, b)


def test_far_elements(nv):
    n = (1 << 32) + 5
    grads = [torch.zeros(n, dtype=BF16, device="cuda")]
    like = nv.adamw_plan([torch.zeros(n, dtype=BF16, device="cuda")], state="e4m3")
    grads[0][-1], grads[0][n // 2], grads[0][0] = 3.0, 4.0, 12.0
    norm, scale = nv.grad_norm(like, grads, max_norm=6.5, eps=0.0)
    assert norm.item() == 13.0 and scale.item() == 0.5
    nv.clip_grads(like, grads, scale)
    assert [grads[0][i].item() for i in (-1, n // 2, 0, 1)] == [1.5, 2.0, 6.0, 0.0]


def test_graphs(nv):
    """Norm and clip captured together on a stream of their own, replayed on other gradients, eager calls
    and synchronizations in between."""
    sizes = [9000, 3, 70_000]
    plan = plan_of(nv, sizes)
    grads = grads_of(sizes, BF16, 0)
    out = [torch.zeros_like(g) for g in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        nv.clip_grads(plan, grads, nv.grad_norm(plan, grads, max_norm=1.0)[1], out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        norm, scale = nv.grad_norm(plan, grads, max_norm=1.0)
        nv.clip_grads(plan, grads, scale, out=out)
    for seed in range(4):
        for g, now in zip(grads, grads_of(sizes, BF16, seed, 0.1 + seed)):
            g.copy_(now)
        graph.replay()
        torch.cuda.synchronize()
        again, by = nv.grad_norm(plan, grads, max_norm=1.0)
        assert torch.equal(norm, again) and torch.equal(scale, by)
        assert all(torch.equal(o, (g.float() * by).to(BF16)) for o, g in zip(out, grads))
        torch.cuda.synchronize()


def test_outputs_of_another_type_than_before(nv):
    """What was recognized for gradients of one type is not taken for those of another."""
    plan, grads = plan_of(nv, [5, 4096, 77]), grads_of([5, 4096, 77], BF16, 3)
    scale = torch.full((1,), 0.5, device="cuda")
    out = [torch.empty_like(g) for g in grads]
    nv.clip_grads(plan, grads, scale, out=out)
    nv.clip_grads(plan, grads, scale, out=out)
    wide = [g.float() for g in grads]
    with pytest.raises(TypeError, match="out must be"):
        nv.clip_grads(plan, wide, scale, out=out)
    to = [torch.empty_like(g) for g in wide]
    for _ in range(2):
        for a, b in zip(nv.clip_grads(plan, wide, scale, out=to), wide):
            assert torch.equal(a, b * 0.5)
    with pytest.raises(TypeError, match="out must be"):
        nv.clip_grads(plan, grads, scale, out=to)


def test_a_bound_of_nothing_for_gradients_of_nothing(nv):
    plan, grads = plan_of(nv, [5, 300]), grads_of([5, 300], F32, 3)
    zeros = [torch.zeros_like(g) for g in grads]
    norm, scale = nv.grad_norm(plan, zeros, max_norm=0.0, eps=0.0)
    assert norm.item() == 0.0 and scale.item() == 1.0


def test_the_same_gradient_twice(nv):
    """Counts twice in the norm; scaled into two outputs."""
    plan = plan_of(nv, [500, 500])
    g = grads_of([500], F32, 3)[0]
    norm, scale = nv.grad_norm(plan, [g, g], max_norm=1.0)
    want = math.sqrt(2 * float(g.double().square().sum()))
    assert close(norm, want)
    out = [torch.zeros_like(g), torch.zeros_like(g)]
    nv.clip_grads(plan, [g, g], scale, out=out)
    assert torch.equal(out[0], g * scale) and torch.equal(out[1], out[0])


def test_refusals(nv):
    plan = plan_of(nv, [8, 9])
    g = [torch.zeros(8, device="cuda"), torch.zeros(9, device="cuda")]
    s, nine, t9 = torch.ones(1, device="cuda"), plan_of(nv, [9, 9]), torch.zeros(9, device="cuda")
    bad = [
        (ValueError, "1 gradients for 2", lambda: nv.grad_norm(plan, g[:1])),
        (ValueError, "gradient 1 is None", lambda: nv.grad_norm(plan, [g[0], None])),
        (ValueError, "8 elements", lambda: nv.grad_norm(plan, [g[1], g[0]])),
        (TypeError, "grads must be", lambda: nv.grad_norm(plan, [g[0], g[1].bfloat16()])),
        (TypeError, "must be bfloat16 or float32", lambda: nv.grad_norm(plan, [t.half() for t in g])),
        (ValueError, "GPU tensors", lambda: nv.grad_norm(plan, [t.cpu() for t in g])),
        (ValueError, "form with max_norm", lambda: nv.grad_norm(plan, g, scale=s)),
        (ValueError, "output must be", lambda: nv.grad_norm(plan, g, norm=s[:0])),
        (ValueError, "workspace", lambda: nv.grad_norm(plan, g, workspace=s)),
        (nv.NVFP4Error, "outside its range", lambda: nv.grad_norm(plan, g, max_norm=-1.0)),
        (nv.NVFP4Error, "outside its range", lambda: nv.grad_norm(plan, g, max_norm=NAN)),
        (nv.NVFP4Error, "outside its range", lambda: nv.grad_norm(plan, g, max_norm=1.0, eps=INF)),
        (nv.NVFP4Error, "overlap", lambda: nv.grad_norm(plan, g, max_norm=1.0, scale=g[0][:1])),
        (TypeError, "scale must be", lambda: nv.clip_grads(plan, g, s.double())),
        (ValueError, "scale must have shape", lambda: nv.clip_grads(plan, g, g[0])),
        (ValueError, "1 outputs for 2", lambda: nv.clip_grads(plan, g, s, out=g[:1])),
        (TypeError, "out must be", lambda: nv.clip_grads(plan, g, s, out=[t.bfloat16() for t in g])),
        (ValueError, "out must be", lambda: nv.clip_grads(plan, g, s, out=[g[1], g[0]])),
        (nv.NVFP4Error, "overlap", lambda: nv.clip_grads(plan, g, g[0][:1])),
        (nv.NVFP4Error, "overlap", lambda: nv.clip_grads(nine, [g[1], g[1]], s)),
        (nv.NVFP4Error, "overlap", lambda: nv.clip_grads(nine, [g[1], g[1].clone()], s, out=[t9, t9])),
        (nv.NVFP4Error, "overlap", lambda: nv.clip_grads(
            plan, [torch.zeros(16, device="cuda")[i:i + n] for i, n in ((0, 8), (0, 9))], g[1][:1], out=g)),
    ]
    for kind, text, call in bad:
        with pytest.raises(kind, match=text):
            call()
