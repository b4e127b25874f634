"""The operators of a quantization-aware distillation step, as measured cases.

Four calls that a training loop makes next to fake-quantization: layer norm forward and
backward, the distillation loss with its gradient, and the AdamW step over many tensors.  Each
case runs either in a plain form (elementary torch operations in 32 bits, rounded once at the
end; ``own = False``) or through this package's calls (``own = True``), on the same inputs.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}

BLOCK = 128             # elements per scale of an 8-bit optimizer state
LR, B1, B2, EPS, WD = 3e-4, 0.9, 0.999, 1e-8, 0.1
NORM_EPS = 1e-5
MASK32 = 0xFFFFFFFF


def listed():
    return [
        # one token of a decode or of a last, short microbatch: launch latency is what counts
        norm("norm_fwd_token", "fwd", 1, 4096, "bf16", "bf16", True, True, False),
        # the activation workload's shape: pre-norm block with residual add, the amax of the
        # output goes to the fake-quantization that follows
        norm("norm_fwd_act", "fwd", 8192, 4096, "bf16", "bf16", True, True, True),
        # rows that are no multiple of a vector, 32-bit activations, root-mean-square form
        norm("norm_fwd_odd_f32", "fwd", 1023, 5119, "f32", "f32", False, False, False),
        # a short microbatch's backward pass
        norm("norm_bwd_small", "bwd", 64, 2048, "bf16", "bf16", True, False, False),
        # the backward pass of norm_fwd_act, with the gradient of the residual stream added
        norm("norm_bwd_act", "bwd", 8192, 4096, "bf16", "bf16", True, True, False),
        # the weight workload's width, 32-bit weights over bf16 activations, odd row count
        norm("norm_bwd_wide", "bwd", 2051, 14336, "bf16", "f32", False, False, False),
        # a few answer tokens: fewer rows than the chip has compute units
        distill("distill_few", 3, 32000, "bf16", 1.0, 0.0, 0),
        # a microbatch of 4096 tokens over a large vocabulary
        distill("distill_large", 4096, 128000, "bf16", 1.0, 0.0, 0),
        # 32-bit logits, odd vocabulary with padded entries, prompt rows without weight
        distill("distill_odd_f32", 515, 50251, "f32", 2.0, 0.25, 11),
        # a small model's tensors, everything in 32 bits
        adamw("adamw_small", "even", 24, 65536, 0, "f32", "f32", False, False, False, False),
        # the 64 experts of the MoE workload: bf16 weights with 32-bit master copies and states;
        # the amax of every new weight goes to its quantization
        adamw("adamw_moe", "even", 64, 2048 * 5120, 0, "bf16", "bf16", True, False, False, True),
        # matrices of many sizes beside vectors, states in 8 bits, no master copy, clipped
        adamw("adamw_8bit", "ragged", 150, 4096 * 14336 * 4, 7, "bf16", "bf16", False, True, True,
              False),
    ]


def norm(name, way, rows, cols, dtype, wdtype, center, residual, amax):
    return {"name": name, "op": "norm", "way": way, "rows": rows, "cols": cols, "dtype": dtype,
            "wdtype": wdtype, "center": center, "residual": residual, "amax": amax}


def distill(name, rows, vocab, dtype, temperature, masked, padded):
    return {"name": name, "op": "distill", "rows": rows, "vocab": vocab, "dtype": dtype,
            "temperature": temperature, "masked": masked, "padded": padded}


def adamw(name, mix, count, most, sizes, dtype, gdtype, master, eight, clip, amax):
    """even: `count` tensors of `most` elements each; ragged: `count` tensors of sizes over a
    wide range (drawn from `sizes`), `most` elements together at the most."""
    return {"name": name, "op": "adamw", "mix": mix, "count": count, "most": most, "sizes": sizes,
            "dtype": dtype, "gdtype": gdtype, "master": master, "eight": eight, "clip": clip,
            "amax": amax}


def spread(rng, lo, hi):
    """lo..hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "distill", "adamw"])
    if op == "norm":
        cols = spread(rng, 256, 16384)
        cols = cols if rng.random() < 0.4 else cols // 64 * 64
        rows = spread(rng, 1, min(16384, 8192 * 4096 // cols))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        way = rng.choice(["fwd", "bwd"])
        c = norm("", way, rows, cols, dtype, rng.choice([dtype, "f32"]), rng.random() < 0.5,
                 rng.random() < 0.5, way == "fwd" and rng.random() < 0.5)
    elif op == "distill":
        vocab = spread(rng, 1000, 200000)
        vocab = vocab if rng.random() < 0.5 else vocab // 64 * 64
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows = spread(rng, 1, min(8192, 4096 * 128000 // vocab // SIZE[dtype]))
        c = distill("", rows, vocab, dtype, rng.choice([1.0, 1.0, 2.0, 0.7]),
                    rng.choice([0.0, 0.25]), rng.choice([0, 0, 37]))
    else:
        eight = rng.random() < 0.5
        dtype = rng.choice(["bf16", "bf16", "f32"])
        count = spread(rng, 1, 300)
        c = adamw("", "ragged", count, spread(rng, 4096 * count, 150_000_000), rng.randrange(1 << 20),
                  dtype, rng.choice(["bf16", "f32"]), dtype == "bf16" and rng.random() < 0.5, eight,
                  rng.random() < 0.5, rng.random() < 0.3)
    del c["name"]
    return c


def tensor_sizes(case):
    """Element counts of an AdamW case's tensors."""
    n, most = case["count"], case["most"]
    if case["mix"] == "even":
        return [most] * n
    rng = random.Random(case["sizes"])
    big = max(1, n // 12)           # few matrices hold most elements, many vectors the rest
    part = [rng.uniform(0.5, 1.5) for _ in range(big)]
    got = [max(1, int(most * 0.95 * p / sum(part))) for p in part]
    return got + [spread(rng, 1, max(2, most // (20 * n))) for _ in range(n - big)]


def work(case):
    if case["op"] == "norm":
        e, w = SIZE[case["dtype"]], SIZE[case["wdtype"]]
        n, cols, rows = case["rows"] * case["cols"], case["cols"], case["rows"]
        stats = 4 * rows * (2 if case["center"] else 1)
        vecs = (2 if case["center"] else 1) * cols * w
        if case["way"] == "fwd":
            return {"bytes": n * e * (4 if case["residual"] else 2) + vecs + stats, "flops": 9 * n}
        return {"bytes": n * e * (4 if case["residual"] else 3) + cols * w + vecs + stats,
                "flops": 14 * n}
    if case["op"] == "distill":
        live = case["rows"] - int(case["rows"] * case["masked"])
        n = case["rows"] * case["vocab"]
        e = SIZE[case["dtype"]]
        return {"bytes": (2 * live * case["vocab"] + n) * e + 8 * case["rows"],
                "flops": 20 * live * case["vocab"]}
    n = sum(tensor_sizes(case))
    state = 4 * (1 + 4 / BLOCK) if case["eight"] else 16
    weight = (SIZE[case["dtype"]] + 8) if case["master"] else 2 * SIZE[case["dtype"]]
    return {"bytes": int(n * (weight + SIZE[case["gdtype"]] + state)), "flops": 16 * n}


# ---------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"norm": prepare_norm, "distill": prepare_distill, "adamw": prepare_adamw}[case["op"]](
        case, gen)


def randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def prepare_norm(case, gen):
    """Residual-stream values: a few channels are far larger than the others, and not centred."""
    rows, cols, T, W = case["rows"], case["cols"], DT[case["dtype"]], DT[case["wdtype"]]
    channel = torch.exp(0.7 * randn(gen, cols))
    s = {"case": case, "x": (randn(gen, rows, cols) * channel + 0.2).to(T),
         "weight": (1 + 0.2 * randn(gen, cols)).to(W),
         "bias": (0.1 * randn(gen, cols)).to(W) if case["center"] else None, "residual": None}
    if case["residual"]:
        s["residual"] = randn(gen, rows, cols).to(T)
    if case["way"] == "bwd":
        s["dy"] = (1e-3 * randn(gen, rows, cols)).to(T)
        if case["residual"]:
            s["residual"] = (1e-3 * randn(gen, rows, cols)).to(T)
        x = s["x"].double()
        mean = x.mean(1, keepdim=True) if case["center"] else 0.0
        s["rstd"] = ((x - mean).square().mean(1) + NORM_EPS).rsqrt().float()
        s["mean"] = mean[:, 0].float() if case["center"] else None
    elif case["amax"]:
        s["amax"] = torch.empty(1, device="cuda")
    return s


def prepare_distill(case, gen):
    """A student near its teacher; padded vocabulary entries at minus infinity."""
    rows, vocab, T = case["rows"], case["vocab"], DT[case["dtype"]]
    t = randn(gen, rows, vocab)
    t.mul_(2.5)
    s = (t + 0.3 * randn(gen, rows, vocab)).to(T)
    t = t.to(T)
    if case["padded"]:
        t[:, -case["padded"]:] = -math.inf
        s[:, -case["padded"]:] = -math.inf
    live = rows - int(rows * case["masked"])
    weight = torch.zeros(rows, device="cuda")
    weight[torch.randperm(rows, generator=gen, device="cuda")[:live]] = 1.0
    weight *= 0.5 + torch.rand(rows, generator=gen, device="cuda")
    return {"case": case, "student": s, "teacher": t, "weight": weight}


def prepare_adamw(case, gen):
    """Parameters, gradients and states in the middle of training: each kind is one buffer
    that the tensors are parts of, every part starting at a multiple of BLOCK elements."""
    sizes = tensor_sizes(case)
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // BLOCK) * BLOCK)
    total = at[-1]
    flat = {"param": torch.zeros(total, dtype=DT[case["dtype"]], device="cuda"),
            "grad": torch.zeros(total, dtype=DT[case["gdtype"]], device="cuda")}
    if case["master"]:
        flat["master"] = torch.zeros(total, device="cuda")
    kind = torch.float8_e4m3fn if case["eight"] else torch.float32
    flat["avg"] = torch.zeros(total, dtype=kind, device="cuda")
    flat["sq"] = torch.zeros(total, dtype=kind, device="cuda")
    if case["eight"]:
        flat["avg_scale"] = torch.zeros(total // BLOCK, device="cuda")
        flat["sq_scale"] = torch.zeros(total // BLOCK, device="cuda")
    part = {k: [f[a // BLOCK:b // BLOCK] if "scale" in k else f[a:a + n]
                for a, b, n in zip(at, at[1:], sizes)] for k, f in flat.items()}
    for k, n in enumerate(sizes):
        size = math.exp(0.5 * (k % 7) - 8)            # gradients of tensors differ in size
        p = 0.02 * randn(gen, n)
        part["param"][k].copy_(p)
        if case["master"]:
            part["master"][k].copy_(part["param"][k].float() + 2e-5 * randn(gen, n))
        del p
        local = torch.exp(randn(gen, n)) * size       # and so do those within one
        part["grad"][k].copy_(local * randn(gen, n))
        avg, sq = 0.3 * local * randn(gen, n), (local * (0.7 + 0.3 * torch.rand(
            n, generator=gen, device="cuda"))).square()
        if case["eight"]:
            for name, x in (("avg", avg), ("sq", sq.sqrt())):
                x = blocks(x)
                scale = x.abs().amax(1) / 448
                part[name + "_scale"][k].copy_(scale)
                part[name][k].copy_((x / scale[:, None]).clamp(-448, 448).reshape(-1)[:n])
        else:
            part["avg"][k].copy_(avg)
            part["sq"][k].copy_(sq)
    s = {"case": case, "flat": flat, "part": part, "seed": 1234, "step": 10,
         "clip": torch.full((1,), 0.37, device="cuda") if case["clip"] else None,
         "amax": torch.zeros(len(sizes), device="cuda") if case["amax"] else None}
    if own:                                            # the optimizer that a program keeps
        import nvfp4_block_scaled_amax_amd as nv
        s["plan"] = nv.adamw_plan(part["param"], part["avg"], part["sq"],
                                  master=part.get("master"), avg_scale=part.get("avg_scale"),
                                  sq_scale=part.get("sq_scale"))
    return s


def blocks(x):
    """A flat tensor as rows of BLOCK elements, the last one filled up with zeros."""
    n = x.numel()
    return torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)


# ---------------------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if case["op"] == "norm":
        if case["way"] == "fwd":
            return norm_forward(s) if own else plain_norm_forward(s)
        return norm_backward(s) if own else plain_norm_backward(s)
    if case["op"] == "distill":
        return distill_loss(s) if own else plain_distill(s)
    if own:
        adamw_step(s)
    else:
        plain_adamw(s)
    out = {k: f for k, f in s["flat"].items() if k != "grad"}
    if s["amax"] is not None:
        out["amax"] = s["amax"]
    return out


def norm_forward(s):
    import nvfp4_block_scaled_amax_amd as nv
    y, h, mean, rstd = nv.layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"],
                                     eps=NORM_EPS, center=s["case"]["center"], amax=s.get("amax"))
    out = {"y": y, "rstd": rstd}
    if s["residual"] is not None:
        out["h"] = h
    if mean is not None:
        out["mean"] = mean
    if "amax" in s:
        out["amax"] = s["amax"]
    return out


def plain_norm_forward(s):
    case, T = s["case"], DT[s["case"]["dtype"]]
    h = s["x"].float()
    if s["residual"] is not None:
        h = (h + s["residual"].float()).to(T).float()
    out, z = {}, h
    if case["center"]:
        mean = h.mean(1)
        z = h - mean[:, None]
        out["mean"] = mean
    rstd = 1 / torch.sqrt(z.square().mean(1) + NORM_EPS)
    y = z * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = y.to(T)
    out.update(y=y, rstd=rstd)
    if s["residual"] is not None:
        out["h"] = h.to(T)
    if "amax" in s:
        out["amax"] = y.abs().amax().float().reshape(1)
    return out


def norm_backward(s):
    import nvfp4_block_scaled_amax_amd as nv
    dx, dw, db = nv.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"],
                                        dres=s["residual"], bias=s["case"]["center"])
    return {"dx": dx, "dw": dw} if db is None else {"dx": dx, "dw": dw, "db": db}


def plain_norm_backward(s):
    case, T, W = s["case"], DT[s["case"]["dtype"]], DT[s["case"]["wdtype"]]
    dy, x = s["dy"].float(), s["x"].float()
    if case["center"]:
        x = x - s["mean"][:, None]
    xh = x * s["rstd"][:, None]
    g = dy * s["weight"].float()
    d = g - xh * (g * xh).mean(1, keepdim=True)
    out = {"dw": (dy * xh).sum(0).to(W)}
    if case["center"]:
        d = d - g.mean(1, keepdim=True)
        out["db"] = dy.sum(0).to(W)
    d = d * s["rstd"][:, None]
    if s["residual"] is not None:
        d = d + s["residual"].float()
    out["dx"] = d.to(T)
    return out


def distill_loss(s):
    import nvfp4_block_scaled_amax_amd as nv
    loss, grad = nv.distill_loss(s["student"], s["teacher"], s["weight"],
                                 temperature=s["case"]["temperature"])
    return {"loss": loss, "grad": grad}


def plain_distill(s):
    """sum p (e^d - 1 - d) with d = log q - log p is the divergence with every term >= 0: the
    direct sum of p (log p - log q) loses the loss of a near student to cancellation."""
    T, weight = s["case"]["temperature"], s["weight"]
    t, q = s["teacher"].float() / T, s["student"].float() / T
    t = t - t.amax(1, keepdim=True)
    t = t - t.exp().sum(1, keepdim=True).log()
    q = q - q.amax(1, keepdim=True)
    q = q - q.exp().sum(1, keepdim=True).log()
    p = t.exp()
    d = q - t
    q = q.exp()
    loss = torch.where(p > 0, p * (torch.expm1(d) - d), q).sum(1)
    grad = (q - p) * (weight / T)[:, None]
    dead = weight == 0
    return {"loss": torch.where(dead, 0.0, weight * loss),
            "grad": torch.where(dead[:, None], 0.0, grad).to(s["student"].dtype)}


def adamw_step(s):
    import nvfp4_block_scaled_amax_amd as nv
    nv.adamw_step(s["plan"], s["part"]["grad"], step=s["step"], lr=LR, betas=(B1, B2), eps=EPS,
                  weight_decay=WD, grad_scale=s["clip"], amax=s["amax"], seed=s["seed"])


def mix32(h):
    """A 32-bit integer hash: two rounds of xor-shift and multiply."""
    h = h ^ (h >> 16)
    h = (h * 0x7FEB352D) & MASK32
    h = h ^ (h >> 15)
    h = (h * 0x846CA68B) & MASK32
    return h ^ (h >> 16)


def random_bits(seed, step, tensor, n):
    """32 random bits per element, from its tensor's key and its place."""
    key = mix32(mix32(mix32(seed) ^ step) ^ tensor)
    return mix32((torch.arange(n, device="cuda") + key) & MASK32)


def down(x, bits, drop):
    """|x| cut to its 32 - drop leading bits after random bits were added below them, with x's
    sign: rounds up as often as the part that is cut off says."""
    word = x.view(torch.int32)
    mag = (word & 0x7FFFFFFF) + bits.int()
    return ((mag & -(1 << drop)) | (word & -0x80000000)).view(torch.float32)


def e4m3(x, bits):
    """Stochastic rounding to E4M3 (3 bits after the leading one, steps of 2^-9 below 2^-6)."""
    mag = x.abs()
    shift = torch.where(mag < 2.0 ** -6, 2.0 ** -6, 0.0)
    return torch.clamp(down(mag + shift, bits, 20) - shift, max=448.0).copysign(x)


def plain_state(x, bits, positive):
    """x in 8 bits with a scale per block -> values (float8), scales."""
    n = x.numel()
    x = blocks(x)
    most = x.abs().amax(1)
    scale = torch.where(most < 2.0 ** -100, 0.0, most * (1 / 448))
    inv = torch.where(scale == 0, 0.0, torch.ones_like(scale) / scale)
    y = e4m3((x * inv[:, None]).reshape(-1)[:n], bits)
    if positive:       # a second moment never becomes zero by rounding: it is divided by
        y = torch.where(x.reshape(-1)[:n] > 0, y.clamp(min=2.0 ** -9), y)
    return y.to(torch.float8_e4m3fn), scale


def plain_adamw(s):
    case, part = s["case"], s["part"]
    t = s["step"]
    rate, root = LR / (1 - B1 ** t), 1 / math.sqrt(1 - B2 ** t)
    for k, param in enumerate(part["param"]):
        n = param.numel()
        g = part["grad"][k].float()
        if s["clip"] is not None:
            g = g * s["clip"]
        avg, sq = part["avg"][k].float(), part["sq"][k].float()
        if case["eight"]:
            avg = (blocks(avg) * part["avg_scale"][k][:, None]).reshape(-1)[:n]
            sq = (blocks(sq) * part["sq_scale"][k][:, None]).reshape(-1)[:n]
            sq = sq * sq
        avg = avg * B1 + g * (1 - B1)
        sq = sq * B2 + (g * g) * (1 - B2)
        low = sq.sqrt()
        p = part["master"][k] if case["master"] else param.float()
        p = p * (1 - LR * WD) - (avg / (low * root + EPS)) * rate
        alone = case["dtype"] == "bf16" and not case["master"]
        bits = random_bits(s["seed"], t, k, n) if case["eight"] or alone else None
        if case["eight"]:
            code, scale = plain_state(avg, bits & 0xFFFFF, False)
            part["avg"][k].copy_(code)
            part["avg_scale"][k].copy_(scale)
            code, scale = plain_state(low, bits >> 12, True)
            part["sq"][k].copy_(code)
            part["sq_scale"][k].copy_(scale)
        else:
            part["avg"][k].copy_(avg)
            part["sq"][k].copy_(sq)
        if case["master"]:
            part["master"][k].copy_(p)
        if alone:
            p = down(p, ((bits * 0x9E3779B1) & MASK32) >> 16, 16)
        param.copy_(p)
        if s["amax"] is not None:
            s["amax"][k] = param.abs().amax()


# ---------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return exact_norm(case, s)
    if case["op"] == "distill":
        return exact_distill(case, s)
    return exact_adamw(case, s)


def exact_norm(case, s):
    h, w = s["x"].double(), s["weight"].double()
    if case["way"] == "fwd":
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(DT[case["dtype"]]).double()
        mean = h.mean(1, keepdim=True) if case["center"] else 0.0
        rstd = ((h - mean).square().mean(1, keepdim=True) + NORM_EPS) ** -0.5
        y = (h - mean) * rstd * w + (s["bias"].double() if case["center"] else 0.0)
        out = {"y": y, "rstd": rstd[:, 0]}
        if s["residual"] is not None:
            out["h"] = h
        if case["center"]:
            out["mean"] = mean[:, 0]
        if case["amax"]:
            out["amax"] = y.abs().amax().reshape(1)
        return out
    # the gradient of sum(y * dy) through the row's statistics, term by term
    cols, dy = case["cols"], s["dy"].double()
    rstd = s["rstd"].double()[:, None]
    xh = (h - (s["mean"].double()[:, None] if case["center"] else 0.0)) * rstd
    up = dy * w
    along = (up * xh).sum(1, keepdim=True) / cols
    level = up.sum(1, keepdim=True) / cols if case["center"] else 0.0
    dx = rstd * (up - level - xh * along)
    if s["residual"] is not None:
        dx = dx + s["residual"].double()
    out = {"dx": dx, "dw": (dy * xh).sum(0)}
    if case["center"]:
        out["db"] = dy.sum(0)
    return out


def exact_distill(case, s):
    T = case["temperature"]
    loss, grad = [], []
    step = max(1, (1 << 27) // case["vocab"])
    for a in range(0, case["rows"], step):
        w = s["weight"][a:a + step].double()
        lp = torch.log_softmax(s["teacher"][a:a + step].double() / T, 1)
        lq = torch.log_softmax(s["student"][a:a + step].double() / T, 1)
        loss.append(w * torch.where(lp > -math.inf, lp.exp() * (lp - lq), 0.0).sum(1))
        grad.append(((lq.exp() - lp.exp()) * (w / T)[:, None]).to(
            torch.float64 if case["rows"] * case["vocab"] < 1 << 28 else torch.float32))
    return {"loss": torch.cat(loss), "grad": torch.cat(grad)}


def exact_adamw(case, s):
    """The update's definition.  Where a value is rounded by random bits (8-bit states, bf16
    parameters without a master copy) it is given before that rounding, which is also the mean
    over all random bits."""
    part, t = s["part"], s["step"]
    held = "master" if case["master"] else "param"
    out = {k: torch.zeros_like(f, dtype=torch.float64) for k, f in s["flat"].items() if k != "grad"}
    top, at = [], 0
    for k, param in enumerate(part["param"]):
        n = param.numel()
        g = part["grad"][k].double()
        if s["clip"] is not None:
            g = g * s["clip"].double()
        m, v = part["avg"][k].double(), part["sq"][k].double()
        if case["eight"]:
            m = m * part["avg_scale"][k].double().repeat_interleave(BLOCK)[:n]
            v = (v * part["sq_scale"][k].double().repeat_interleave(BLOCK)[:n]) ** 2
        m, v = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g * g
        hat = (m / (1 - B1 ** t)) / ((v / (1 - B2 ** t)) ** 0.5 + EPS)
        p = part[held][k].double()
        p = p - LR * (hat + WD * p)
        for name, x in (("param", p), ("master", p), ("avg", m), ("sq", v)):
            if case["eight"] and name in ("avg", "sq"):
                x = x if name == "avg" else x ** 0.5
                scale = blocks(x).abs().amax(1) / 448
                x = x / scale.clamp(min=1e-300).repeat_interleave(BLOCK)[:n]
                out[name + "_scale"][at // BLOCK:at // BLOCK + scale.numel()] = scale
            if name in out:
                out[name][at:at + n] = x
        top.append(p.abs().amax())
        at += -(-n // BLOCK) * BLOCK
    if s["amax"] is not None:
        out["amax"] = torch.stack(top)
    return out
