"""Products of a few rows with packed weights against 64 bits (GPU).

Most cases are made so that every partial sum is a number that binary32 holds, whatever the order:
x and the weights are small multiples of fixed units.  Then the sum is exact and y is known to the bit: one
product with alpha and one rounding.  Values of ordinary size get the bound of a sum of `cols` terms."""
from __future__ import annotations

import ctypes
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)


@pytest.fixture(scope="module")
def nv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import nvfp4_block_scaled_amax_amd as m
    m.lib()
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def weights(shape, seed, scale_bytes=(0x38, 0x48)):
    """Random codes, and scales of 1 to 3.75 in steps of 1/8 or 1/4 -> codes, scales, alpha, values."""
    g = gen(seed)
    E, rows, cols = shape
    code = torch.randint(0, 16, (E, rows, cols), generator=g, dtype=torch.int64)
    scale = torch.randint(*scale_bytes, (E, rows, cols // 16), generator=g, dtype=torch.int64).to(torch.uint8)
    codes = (code[..., 0::2] | code[..., 1::2] << 4).to(torch.uint8)
    alpha = torch.rand(E, generator=g) + 0.01
    value = E2M1[code] * scale.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    return codes, scale, alpha, value


def rounded(total, alpha, dtype):
    """The exact sums (multiples of 1/16 below 2^20) times alpha, rounded."""
    assert total.abs().max() < 2 ** 20
    return (total.float() * alpha).to(dtype)


def whole(shape, seed, most=4):
    return torch.randint(-most, most + 1, shape, generator=gen(seed)).float()


def same(a, b):
    return torch.equal(a.cpu().view(torch.int16 if a.dtype == BF16 else torch.int32),
                       b.view(torch.int16 if b.dtype == BF16 else torch.int32))


SHAPES = [(1, 1, 16), (1, 256, 256), (1, 16, 128), (2, 17, 144), (3, 33, 272), (5, 100, 1008),
          (6, 47, 2064), (7, 31, 4080), (8, 64, 112), (16, 256, 1024), (17, 130, 1040), (32, 65, 528),
          (33, 200, 624), (64, 48, 2048), (65, 16, 144), (100, 129, 272), (1, 4099, 14336), (13, 1000, 5104)]


@pytest.mark.parametrize("xtype,ytype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("tokens,rows,cols", SHAPES)
def test_exact_sums(nv, tokens, rows, cols, xtype, ytype):
    codes, scales, alpha, value = weights((1, rows, cols), tokens + rows)
    x = whole((tokens, cols), cols)
    want = rounded(x.double() @ value[0].t(), alpha, ytype)
    got = nv.packed_matvec(x.to(xtype).cuda(), codes[0].cuda(), scales[0].cuda(), alpha.cuda(), dtype=ytype)
    assert got.shape == (tokens, rows) and got.dtype == ytype
    assert same(got, want)


@pytest.mark.parametrize("xtype", [BF16, F32])
@pytest.mark.parametrize("tokens,rows,cols", [(1, 32801, 1040), (4, 130, 2000), (8, 90, 4112), (4, 70, 2576),
                                              (20, 8211, 1040), (7, 8211, 1040), (9, 61, 12304),
                                              (40, 8211, 1040), (300, 130, 496), (1024, 70, 1040), (1000, 33, 4112),
                                              (64, 515, 8208), (100, 2000, 4112), (90, 4100, 1552), (40, 515, 8208),
                                              (12, 1000, 4112), (70, 12290, 528)])
def test_exact_sums_of_more_sizes(nv, tokens, rows, cols, xtype):
    test_exact_sums(nv, tokens, rows, cols, xtype, F32)


@pytest.mark.parametrize("bits", [9, 16, 17, 24])
def test_every_bit_of_32_bit_rows_counts(nv, bits):
    """x of up to 24 significant bits against one weight of 1 per row: y is x."""
    cols = 256
    x = (torch.randint(1 << (bits - 1), 1 << bits, (3, cols), generator=gen(bits)).double()
         * torch.where(torch.rand(3, cols, generator=gen(1)) < 0.5, -1.0, 1.0)).float()
    x *= torch.exp2(torch.randint(-60, 60, (3, cols), generator=gen(2)).float())
    code = torch.zeros(cols, cols, dtype=torch.int64)
    code[torch.arange(cols), torch.arange(cols)] = 2                    # 1.0
    codes = (code[:, 0::2] | code[:, 1::2] << 4).to(torch.uint8)
    scales = torch.full((cols, cols // 16), 0x38, dtype=torch.uint8)
    got = nv.packed_matvec(x.cuda(), codes.cuda(), scales.cuda(), torch.ones(1).cuda())
    assert same(got, x)


@pytest.mark.parametrize("tokens", [1, 7])
@pytest.mark.parametrize("power", [-100, -110, -111, -120, -126, -133, -140])
def test_small_32_bit_rows(nv, tokens, power):
    """x of 24 significant bits against one weight of 1 per row, and an alpha that brings the sums back: what x
    has below 2^-133, the smallest bf16, is cut off, and nothing else."""
    cols = 256
    x = torch.randint(1 << 23, 1 << 24, (tokens, cols), generator=gen(1)).double() * 2.0 ** (power - 23)
    x = x.float()
    code = torch.zeros(cols, cols, dtype=torch.int64)
    code[torch.arange(cols), torch.arange(cols)] = 2                    # 1.0
    codes = (code[:, 0::2] | code[:, 1::2] << 4).to(torch.uint8)
    scales = torch.full((cols, cols // 16), 0x38, dtype=torch.uint8)
    got = nv.packed_matvec(x.cuda(), codes.cuda(), scales.cuda(), torch.full((1,), 2.0 ** 100).cuda())
    off = (x.double() - got.cpu().double() * 2.0 ** -100).abs()
    assert (off < 2.0 ** -133).all() and (power < -110 or not off.any())


@pytest.mark.parametrize("picks,itype,tokens,E,rows,cols", [
    (None, torch.int64, 9, 4, 40, 144), (1, torch.int32, 1, 8, 33, 272), (2, torch.int32, 5, 3, 64, 128),
    (4, torch.int64, 24, 16, 100, 1024), (8, torch.int64, 128, 64, 48, 96), (3, torch.int32, 40, 2, 17, 400)])
@pytest.mark.parametrize("xtype,ytype", [(BF16, BF16), (F32, F32)])
def test_experts(nv, picks, itype, tokens, E, rows, cols, xtype, ytype):
    """Each token's experts, the same expert for many tokens or twice for one, experts without a token,
    and indices that are none: these rows are zero."""
    codes, scales, alpha, value = weights((E, rows, cols), tokens)
    x = whole((tokens, cols), 5)
    shape = (tokens,) if picks is None else (tokens, picks)
    expert = torch.randint(0, E, shape, generator=gen(3)).to(itype)
    flat = expert.view(-1)
    if flat.numel() > 3:
        flat[0], flat[flat.numel() // 2], flat[-1] = -1, E, torch.iinfo(itype).min
    k = picks or 1
    want = torch.zeros(tokens * k, rows, dtype=ytype)
    for i, e in enumerate(flat.tolist()):
        if 0 <= e < E:
            want[i] = rounded(value[e] @ x[i // k].double(), alpha[e], ytype)
    y = torch.full(shape + (rows,), float("nan"), dtype=ytype, device="cuda")
    got = nv.packed_matvec(x.to(xtype).cuda(), codes.cuda(), scales.cuda(), alpha.cuda(),
                           expert=expert.cuda(), dtype=ytype, y=y)
    assert got is y
    assert same(got.view(tokens * k, rows), want)


@pytest.mark.parametrize("picks,tokens,E,rows,cols", [
    (4, 60, 3, 40, 1552), (2, 12, 16, 70, 1008), (2, 20, 5, 100, 2064), (1, 14, 5, 50, 5136), (2, 3, 8, 100, 4112),
    (1, 9, 9, 33, 10848), (1, 12, 8, 50, 1552), (1, 12, 64, 20, 1552), (2, 10, 5, 60, 4112), (1, 8, 10, 47, 8176),
    (1, 7, 8, 8003, 1040), (1, 7, 64, 20, 1552), (2, 100, 4, 130, 1552),
    (8, 128, 16, 64, 2576), (1, 1000, 3, 40, 4112), (4, 200, 8, 33, 400), (3, 90, 6, 3001, 1040),
    (2, 24, 6, 1700, 2576)])
@pytest.mark.parametrize("one", [False, True])
@pytest.mark.parametrize("xtype,ytype", [(BF16, F32), (F32, BF16)])
def test_experts_of_long_rows(nv, picks, tokens, E, rows, cols, one, xtype, ytype):
    """Rows of several units; every token at the same expert, which is more than its share."""
    codes, scales, alpha, value = weights((E, rows, cols), tokens)
    x = whole((tokens, cols), 5)
    expert = torch.full((tokens, picks), E // 2) if one else torch.randint(0, E, (tokens, picks), generator=gen(3))
    want = torch.empty(tokens, picks, rows, dtype=ytype)
    for e in expert.unique().tolist():
        at = (expert == e).nonzero()
        want[at[:, 0], at[:, 1]] = rounded(x[at[:, 0]].double() @ value[e].t(), alpha[e], ytype)
    got = nv.packed_matvec(x.to(xtype).cuda(), codes.cuda(), scales.cuda(), alpha.cuda(), expert=expert.cuda(),
                           dtype=ytype)
    assert same(got, want)


def test_no_row_has_an_expert(nv):
    codes, scales, alpha, _ = weights((3, 20, 64), 0)
    y = torch.ones(4, 20, dtype=BF16, device="cuda")
    nv.packed_matvec(torch.ones(4, 64, dtype=BF16, device="cuda"), codes.cuda(), scales.cuda(),
                     alpha.cuda(), expert=torch.full((4,), -1, device="cuda"), y=y)
    assert not y.any()


@pytest.mark.parametrize("tokens", [0, 1, 3])
def test_nothing_beside_the_outputs_is_written(nv, tokens):
    rows, cols = 37, 144
    codes, scales, alpha, value = weights((1, rows, cols), 1)
    for xtype in (BF16, F32):
        x = whole((tokens, cols), 2)
        held = torch.full((tokens * rows + 64,), 7.0, device="cuda")
        y = held[32:32 + tokens * rows].view(tokens, rows)
        nv.packed_matvec(x.to(xtype).cuda(), codes[0].cuda(), scales[0].cuda(), alpha.cuda(), dtype=F32, y=y)
        assert (held[:32] == 7).all() and (held[32 + tokens * rows:] == 7).all()
        if tokens:
            assert same(y, rounded(x.double() @ value[0].t(), alpha, F32))


@pytest.mark.parametrize("xtype", [BF16, F32])
def test_strides_and_odd_starts(nv, xtype):
    """Rows of x apart and at odd elements, codes at 8 bytes past a 16-byte boundary, scales and the
    rows of weights at odd addresses."""
    rows, cols = 21, 400                                  # 200 bytes of codes, 25 of scales a row
    codes, scales, alpha, value = weights((1, rows, cols), 4)
    x = whole((5, cols), 6)
    wide = torch.full((5, cols + 31), float("nan"), dtype=xtype, device="cuda")
    wide[:, 3:3 + cols] = x.to(xtype)
    c = torch.zeros(rows * cols // 2 + 16, dtype=torch.uint8, device="cuda")[8:8 + rows * cols // 2]
    s = torch.zeros(rows * cols // 16 + 9, dtype=torch.uint8, device="cuda")[3:3 + rows * cols // 16]
    c.copy_(codes[0].reshape(-1))
    s.copy_(scales[0].reshape(-1))
    got = nv.packed_matvec(wide[:, 3:3 + cols], c.view(rows, -1), s.view(rows, -1), alpha.cuda(), dtype=F32)
    assert same(got, rounded(x.double() @ value[0].t(), alpha, F32))


def test_leading_dimensions_and_a_single_row(nv):
    codes, scales, alpha, value = weights((1, 30, 96), 4)
    args = codes[0].cuda(), scales[0].cuda(), alpha.cuda()
    x = whole((2, 3, 96), 6)
    want = rounded(x.double() @ value[0].t(), alpha, BF16)
    assert same(nv.packed_matvec(x.to(BF16).cuda(), *args), want)
    assert same(nv.packed_matvec(x[1, 2].to(BF16).cuda(), *args), want[1, 2])
    assert nv.packed_matvec(x[:0].to(BF16).cuda(), *args).shape == (0, 3, 30)


@pytest.mark.parametrize("cols", [64, 1040])
@pytest.mark.parametrize("xtype", [BF16, F32])
def test_values_that_are_not_finite(nv, xtype, cols):
    """An infinity times a positive, a negative and a zero weight; a NaN; a NaN scale; a NaN alpha: only
    the outputs that they belong to."""
    code = torch.full((5, cols), 2, dtype=torch.int64)
    code[1], code[2] = 10, 0                              # 1, -1, 0, 1, 1
    codes = (code[:, 0::2] | code[:, 1::2] << 4).to(torch.uint8)
    scales = torch.full((5, cols // 16), 0x38, dtype=torch.uint8)
    scales[3, cols // 16 - 1] = 0x7F
    x = torch.ones(4, cols)
    x[1, cols - 1], x[2, 0], x[3, 5] = float("inf"), float("nan"), float("-inf")
    got = nv.packed_matvec(x.to(xtype).cuda(), codes.cuda(), scales.cuda(), torch.ones(1).cuda()).float().cpu()
    inf, nan = float("inf"), float("nan")
    n = float(torch.tensor(float(cols)).to(xtype))
    want = torch.tensor([[n, -n, 0, nan, n], [inf, -inf, nan, nan, inf], [nan] * 5, [-inf, inf, nan, nan, -inf]])
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(1e9), want.nan_to_num(1e9))
    got = nv.packed_matvec(x.to(xtype).cuda(), codes.cuda(), scales.cuda(), torch.full((1,), nan).cuda())
    assert torch.isnan(got).all()


@pytest.mark.parametrize("mode", ["rtn6", "four_over_six"])
@pytest.mark.parametrize("tokens,rows,cols", [(1, 300, 4096), (4, 1000, 1504), (20, 515, 2048)])
@pytest.mark.parametrize("xtype", [BF16, F32])
def test_quantized_weights(nv, xtype, tokens, rows, cols, mode):
    """Weights from quantize().  The sum of `cols` terms is off by at most cols steps of its terms'
    sum of magnitudes (2^-23: a matrix instruction may cut instead of round), alpha and the result are
    rounded once each."""
    w = (0.02 * torch.randn(rows, cols, generator=gen(1))).to(BF16)
    codes, scales, alpha = nv.quantize(w.cuda(), mode)
    x = torch.randn(tokens, cols, generator=gen(2)).to(xtype)
    got = nv.packed_matvec(x.cuda(), codes, scales, alpha, dtype=F32).cpu().double()
    c = codes.cpu().long()
    value = E2M1[torch.stack((c & 15, c >> 4), 2).view(rows, cols)]
    value = value * scales.cpu().view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * alpha.item()
    want, size = x.double() @ value.t(), x.double().abs() @ value.abs().t()
    off = (got - want).abs()
    assert (off <= cols * 2.0 ** -23 * size + 2.0 ** -23 * want.abs()).all()
    # the errors' own size: rounding is not one-sided by more than a few steps of the result
    assert off.norm() <= 2.0 ** -18 * size.norm()
    # and the packed weight is the one that dequantize gives (rounded to bf16 there)
    full = x.cuda().float() @ nv.dequantize(codes, scales, alpha).float().t()
    assert (full.cpu().double() - want).norm() <= 2.0 ** -8 * want.norm()


def test_far_weights(nv):
    """An expert behind the first 2^31 bytes of codes, and its scales behind 2^28."""
    E, rows, cols = 70, 8192, 8192
    codes = torch.zeros(E, rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(E, rows, cols // 16, dtype=torch.uint8, device="cuda")
    c, s, alpha, value = weights((1, 64, cols), 9)
    codes[-1, -64:], scales[-1, -64:] = c[0].cuda(), s[0].cuda()
    x = whole((2, cols), 2, most=2)
    y = nv.packed_matvec(x.to(BF16).cuda(), codes, scales, alpha.cuda().repeat(E),
                         expert=torch.tensor([E - 1, 0], device="cuda"), dtype=F32)
    assert same(y[0, -64:], rounded(value[0] @ x[0].double(), alpha, F32))
    assert not y[0, :-64].any() and not y[1].any()


@pytest.mark.parametrize("xtype", [BF16, F32])
def test_graphs_and_streams(nv, xtype):
    """Captured on a stream of its own and replayed with other inputs, eager calls in between; the same
    bits each time."""
    rows, cols = 200, 528
    codes, scales, alpha, value = weights((4, rows, cols), 1)
    args = codes.cuda(), scales.cuda(), alpha.cuda()
    x, expert = torch.zeros(6, cols, dtype=xtype, device="cuda"), torch.zeros(6, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        nv.packed_matvec(x, *args, expert=expert)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = nv.packed_matvec(x, *args, expert=expert)
    for seed in range(4):
        now, ids = whole((6, cols), seed), torch.randint(0, 4, (6,), generator=gen(seed))
        x.copy_(now)
        expert.copy_(ids)
        graph.replay()
        eager = nv.packed_matvec(x, *args, expert=expert)
        torch.cuda.synchronize()
        want = torch.stack([rounded(value[e] @ v.double(), alpha[e], xtype) for e, v in zip(ids, now)])
        assert same(y, want) and same(eager, want)


@pytest.mark.parametrize("xtype", [BF16, F32])
@pytest.mark.parametrize("tokens,rows,cols", [(1, 300, 14336), (16, 200, 5120), (40, 700, 4112), (20, 9000, 1040)])
def test_a_graph_of_more_shared_memory(nv, tokens, rows, cols, xtype):
    """The forms that ask for more shared memory than a launch gets by itself, first called within a capture."""
    codes, scales, alpha, value = weights((1, rows, cols), 1)
    args = codes[0].cuda(), scales[0].cuda(), alpha.cuda()
    x, graph = torch.zeros(tokens, cols, dtype=xtype, device="cuda"), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = nv.packed_matvec(x, *args)
    for seed in range(3):
        now = whole((tokens, cols), seed)
        x.copy_(now)
        graph.replay()
        eager = nv.packed_matvec(x, *args)
        torch.cuda.synchronize()
        want = rounded(now.double() @ value[0].t(), alpha, xtype)
        assert same(y, want) and same(eager, want)


def test_two_streams_at_once(nv):
    """Calls on two streams that overlap: each has the result it has alone."""
    codes, scales, alpha, value = weights((1, 4099, 2064), 1)
    args = codes[0].cuda(), scales[0].cuda(), alpha.cuda()
    inputs = [whole((t, 2064), t) for t in (1, 7, 16, 33)]
    there = [x.to(BF16).cuda() for x in inputs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        with torch.cuda.stream(streams[i % 2]):
            got.append(nv.packed_matvec(there[(i // 2) % 4], *args, dtype=F32))
    torch.cuda.synchronize()
    want = [rounded(x.double() @ value[0].t(), alpha, F32) for x in inputs]
    for i, y in enumerate(got):
        assert same(y, want[(i // 2) % 4])


class KernelNode(ctypes.Structure):
    """hipKernelNodeParams."""
    _fields_ = [("block", ctypes.c_uint * 3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p),
                ("grid", ctypes.c_uint * 3), ("params", ctypes.c_void_p), ("shared", ctypes.c_uint)]


def launch_of(call):
    """Grid and bytes of shared memory of the one kernel that a call launches, from a capture of it."""
    hip = ctypes.CDLL("libamdhip64.so")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    raw, count = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(1)
    node, got = (ctypes.c_void_p * 1)(), KernelNode()
    assert hip.hipGraphGetNodes(raw, None, ctypes.byref(count)) == 0 and count.value == 1
    assert hip.hipGraphGetNodes(raw, node, ctypes.byref(count)) == 0
    assert hip.hipGraphKernelNodeGetParams(ctypes.c_void_p(node[0]), ctypes.byref(got)) == 0
    return tuple(got.grid), got.shared


@pytest.mark.parametrize("tokens,rows,cols,xtype,passes", [
    (4, 4096, 1536, BF16, 1), (4, 2048, 2560, BF16, 1), (4, 4096, 3584, BF16, 1), (8, 4096, 2560, BF16, 1),
    (8, 4096, 5120, BF16, 1), (16, 8960, 1536, BF16, 1), (16, 8960, 2560, BF16, 1), (16, 1024, 2560, BF16, 2),
    (24, 14336, 1536, BF16, 1), (1, 4096, 2560, F32, 1), (5, 1024, 2560, F32, 3)])
def test_columns_that_fit_go_at_once(nv, tokens, rows, cols, xtype, passes):
    """Rows of x that a workgroup has room for, of lengths that are no power of two of units: as few passes, each of
    which reads the weights, as the columns of the form make (1024 weight rows take the form of 8 columns: two
    passes for 16 of bf16, three for 5 rows of binary32, three columns each).  Passes go side by side, a layer
    of the grid each."""
    codes, scales, alpha, value = weights((1, rows, cols), 2)
    x, args = whole((tokens, cols), 3), (codes[0].cuda(), scales[0].cuda(), alpha.cuda())
    there = x.to(xtype).cuda()
    got = nv.packed_matvec(there, *args, dtype=F32)
    assert same(got, rounded(x.double() @ value[0].t(), alpha, F32))
    grid, shared = launch_of(lambda: nv.packed_matvec(there, *args, dtype=F32, y=got))
    assert grid[1:] == (1, passes), (grid, shared)


def test_two_threads_at_once(nv):
    """Calls of two threads of one form with more shared memory than a launch gets by itself, of different sizes."""
    codes, scales, alpha, value = weights((1, 96, 14336), 1)
    inputs = [whole((t, 14336), t) for t in (1, 2, 3, 4)]
    there = [x.to(BF16).cuda() for x in inputs]
    args = codes[0].cuda(), scales[0].cuda(), alpha.cuda()
    got = [[], []]

    def calls(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            for i in range(200):
                got[k].append(nv.packed_matvec(there[2 * (i % 2) + k], *args, dtype=F32))
    torch.cuda.synchronize()
    threads = [threading.Thread(target=calls, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    want = [rounded(x.double() @ value[0].t(), alpha, F32) for x in inputs]
    for k in range(2):
        assert len(got[k]) == 200
        for i, y in enumerate(got[k]):
            assert same(y, want[2 * (i % 2) + k])


def test_refusals(nv):
    codes, scales, alpha, _ = weights((2, 32, 64), 0)
    c, s, a = codes.cuda(), scales.cuda(), alpha.cuda()
    x = torch.ones(3, 64, dtype=BF16, device="cuda")
    one = c[0], s[0], a[:1]
    e = torch.zeros(3, dtype=torch.int64, device="cuda")
    bad = [
        (TypeError, "x must be", lambda: nv.packed_matvec(x.half(), *one)),
        (TypeError, "scales must be", lambda: nv.packed_matvec(x, c[0], s[0].float(), a[:1])),
        (TypeError, "dtype", lambda: nv.packed_matvec(x, *one, dtype=torch.float16)),
        (ValueError, "codes must be", lambda: nv.packed_matvec(x, c, s, a)),
        (ValueError, "codes must be", lambda: nv.packed_matvec(x, *one, expert=e)),
        (ValueError, "codes must have shape", lambda: nv.packed_matvec(x[:, :48], *one)),
        (ValueError, "multiple of 16", lambda: nv.packed_matvec(x[:, :40], *one)),
        (ValueError, "at least 1", lambda: nv.packed_matvec(x[:, :0].contiguous(), c[0, :, :0].contiguous(),
                                                            s[0, :, :0].contiguous(), a[:1])),
        (ValueError, "alpha must have shape", lambda: nv.packed_matvec(x, c[0], s[0], a)),
        (ValueError, "scales must have shape", lambda: nv.packed_matvec(x, c[0], s[0, :31], a[:1])),
        (ValueError, "contiguous", lambda: nv.packed_matvec(x, c[0].t().contiguous().t(), s[0], a[:1])),
        (ValueError, "contiguous", lambda: nv.packed_matvec(x.t().contiguous().t(), *one)),
        (ValueError, "on cuda", lambda: nv.packed_matvec(x, c[0].cpu(), s[0], a[:1])),
        (ValueError, "expert must be", lambda: nv.packed_matvec(x, c, s, a, expert=e[:2])),
        (TypeError, "expert must be", lambda: nv.packed_matvec(x, c, s, a, expert=e.float())),
        (ValueError, "tokens, cols", lambda: nv.packed_matvec(x[None], c, s, a, expert=e)),
        (ValueError, "at most 1024", lambda: nv.packed_matvec(x[:1].expand(1025, 64).contiguous(), *one)),
        (ValueError, "output must be", lambda: nv.packed_matvec(x, *one, y=torch.empty(3, 32, device="cuda"))),
        (nv.NVFP4Error, "overlap", lambda: nv.packed_matvec(
            x, *one, y=x.view(-1)[:96].view(3, 32))),
    ]
    for kind, text, call in bad:
        with pytest.raises(kind, match=text):
            call()
