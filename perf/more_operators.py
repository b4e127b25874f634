"""The operators of a training step on a model's own answers, as measured cases.

Products of a few rows with packed NVFP4 weights (the answers), log probabilities of given tokens
with entropy and top alternatives, forward and backward (their scores and the loss on them), and the
global gradient norm with clipping (the update).  Each case runs either in a plain form (elementary
torch operations in 32 bits, rounded once at the end; ``own = False``) or through this package's
calls (``own = True``), on the same inputs.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}

BLOCK = 16              # elements per E4M3 scale of a packed weight
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
MOST = 6.0 * 448.0      # the largest value of a code times the largest of a scale
CLIP_EPS = 1e-6


def listed():
    return [
        # one token of one answer through the weight workload's matrix: its largest reads are one
        # byte per 1.8 weights, and it is over in microseconds
        matvec("matvec_token", 1, 4096, 14336, 0, 0, 0, "bf16", "bf16"),
        # sixteen answers at once, the other way through a layer of those widths
        matvec("matvec_batch", 16, 14336, 4096, 0, 0, 0, "bf16", "bf16"),
        # the MoE workload's experts: 24 tokens go to 4 experts each, which hit 44 of the 64
        matvec("matvec_moe", 24, 2048, 5120, 64, 4, 44, "bf16", "bf16"),
        # logits of an odd vocabulary in 32 bits, a width of 255 blocks
        matvec("matvec_odd_f32", 7, 50251, 4080, 0, 0, 0, "f32", "f32"),
        # the token just drawn, with its 20 alternatives: fewer rows than compute units
        logprobs("logp_token", "fwd", 1, 128000, "bf16", 1, 20, 0.8, 0.0, 0),
        # scoring a microbatch of answers, 20 alternatives kept for each token
        logprobs("logp_large", "fwd", 4096, 128000, "bf16", 1, 20, 1.0, 0.0, 0),
        # a student's log probabilities of a teacher's 20 saved alternatives, 32-bit logits, odd
        # vocabulary with padded entries, prompt rows without a token
        logprobs("logp_odd_f32", "fwd", 515, 50251, "f32", 20, 0, 1.0, 0.25, 11),
        # the gradient of logp_large's scores, with an entropy bonus
        logprobs("logp_bwd_large", "bwd", 4096, 128000, "bf16", 1, 0, 1.0, 0.0, 0),
        # the gradient of logp_odd_f32's
        logprobs("logp_bwd_odd_f32", "bwd", 515, 50251, "f32", 20, 0, 1.0, 0.25, 11),
        # a small model's tensors in 32 bits
        norm("norm_small", "norm", "even", 24, 65536, 0, "f32"),
        # matrices of many sizes beside vectors
        norm("norm_ragged", "norm", "ragged", 150, 4096 * 14336 * 4, 7, "bf16"),
        # the gradients of the MoE workload's 64 experts, scaled to the largest norm allowed; they go to
        # buffers of their own here so that a pass can be repeated
        norm("clip_moe", "clip", "even", 64, 2048 * 5120, 0, "bf16"),
    ]


def matvec(name, rows, n, k, experts, picks, hit, dtype, out):
    """experts = 0: one matrix [n, k].  Otherwise [experts, n, k]: each row of x goes to `picks`
    experts, `hit` different ones over all rows."""
    return {"name": name, "op": "matvec", "rows": rows, "n": n, "k": k, "experts": experts,
            "picks": picks, "hit": hit, "dtype": dtype, "out": out}


def logprobs(name, way, rows, vocab, dtype, given, top, temperature, masked, padded):
    return {"name": name, "op": "logprobs", "way": way, "rows": rows, "vocab": vocab, "dtype": dtype,
            "given": given, "top": top, "temperature": temperature, "masked": masked,
            "padded": padded}


def norm(name, way, mix, count, most, sizes, dtype):
    """even: `count` tensors of `most` elements each; ragged: `count` tensors of sizes over a
    wide range (drawn from `sizes`), `most` elements together at the most."""
    return {"name": name, "op": "norm", "way": way, "mix": mix, "count": count, "most": most,
            "sizes": sizes, "dtype": dtype}


def spread(rng, lo, hi):
    """lo..hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["matvec", "matvec", "logprobs", "logprobs", "norm"])
    if op == "matvec":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        out = rng.choice([dtype, "f32"])
        k = BLOCK * spread(rng, 16, 1024)
        if rng.random() < 0.4:
            experts, picks = rng.choice([8, 16, 32, 64]), rng.choice([1, 2, 4, 8])
            rows = spread(rng, 1, 64)
            n = spread(rng, 256, max(256, min(8192, 64 * 2048 * 5120 // (k * experts))))
            hit = rng.randint(picks, min(experts, rows * picks))
        else:
            rows, experts, picks, hit = spread(rng, 1, 64), 0, 0, 0
            n = spread(rng, 256, min(131072, 50251 * 8160 // k))
        c = matvec("", rows, n, k, experts, picks, hit, dtype, out)
    elif op == "logprobs":
        vocab = spread(rng, 1000, 200000)
        vocab = vocab if rng.random() < 0.5 else vocab // 64 * 64
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows = spread(rng, 1, min(8192, 4096 * 128000 // vocab // SIZE[dtype]))
        way = rng.choice(["fwd", "bwd"])
        c = logprobs("", way, rows, vocab, dtype, rng.choice([1, 1, 8, 20, 64]),
                     rng.choice([0, 1, 5, 20, 64]) if way == "fwd" else 0, rng.choice([1.0, 1.0, 2.0, 0.7]),
                     rng.choice([0.0, 0.25]), rng.choice([0, 0, 37]))
    else:
        count = spread(rng, 1, 300)
        c = norm("", rng.choice(["norm", "clip"]), "ragged", count, spread(rng, 4096 * count, 300_000_000),
                 rng.randrange(1 << 20), rng.choice(["bf16", "f32"]))
    del c["name"]
    return c


def tensor_sizes(case):
    """Element counts of a gradient-norm case's tensors."""
    n, most = case["count"], case["most"]
    if case["mix"] == "even":
        return [most] * n
    rng = random.Random(case["sizes"])
    big = max(1, n // 12)           # few matrices hold most elements, many vectors the rest
    part = [rng.uniform(0.5, 1.5) for _ in range(big)]
    got = [max(1, int(most * 0.95 * p / sum(part))) for p in part]
    return got + [spread(rng, 1, max(2, most // (20 * n))) for _ in range(n - big)]


def work(case):
    if case["op"] == "matvec":
        n, k = case["n"], case["k"]
        out = case["rows"] * max(1, case["picks"])
        held = max(1, case["hit"]) * n * k
        return {"bytes": held // 2 + held // BLOCK + case["rows"] * k * SIZE[case["dtype"]]
                + out * n * SIZE[case["out"]] + 4 * out, "flops": 2 * out * n * k}
    if case["op"] == "logprobs":
        live = case["rows"] - int(case["rows"] * case["masked"])
        e, vocab = SIZE[case["dtype"]], case["vocab"]
        small = case["rows"] * (12 * case["given"] + 12 * case["top"] + 12)
        if case["way"] == "fwd":
            return {"bytes": live * vocab * e + small, "flops": 8 * live * vocab}
        return {"bytes": (live + case["rows"]) * vocab * e + small, "flops": 8 * live * vocab}
    n = sum(tensor_sizes(case))
    e = SIZE[case["dtype"]]
    return {"bytes": n * e * (1 if case["way"] == "norm" else 2) + 8,
            "flops": n * (2 if case["way"] == "norm" else 3)}


# ---------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"matvec": prepare_matvec, "logprobs": prepare_logprobs, "norm": prepare_norm}[case["op"]](
        case, gen, seed)


def randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def pack(w):
    """[n, k] values of a weight -> codes, scales, alpha: every block's largest becomes 6 * scale."""
    n, k = w.shape
    alpha = w.abs().amax().reshape(1) / MOST
    w = w.view(n, k // BLOCK, BLOCK)
    scale = (w.abs().amax(2) / (6 * alpha)).to(torch.float8_e4m3fn)
    v = w / (scale.float() * alpha).clamp(min=1e-30)[:, :, None]
    edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(v.abs(), edge, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    code = code.view(n, k // 2, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4), scale.view(torch.uint8), alpha


def prepare_matvec(case, gen, seed):
    """Weights of a normal distribution, of another size in each expert; activations whose channels
    differ in size."""
    rows, n, k, E = case["rows"], case["n"], case["k"], case["experts"]
    codes = torch.empty(max(E, 1), n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(max(E, 1), n, k // BLOCK, dtype=torch.uint8, device="cuda")
    alpha = torch.empty(max(E, 1), device="cuda")
    for e in range(max(E, 1)):
        size = 0.02 * math.exp(0.2 * (e % 7))
        codes[e], scales[e], alpha[e:e + 1] = pack(size * randn(gen, n, k))
    x = (randn(gen, rows, k) * torch.exp(0.7 * randn(gen, k))).to(DT[case["dtype"]])
    s = {"case": case, "x": x, "codes": codes if E else codes[0], "scales": scales if E else scales[0],
         "alpha": alpha, "expert": None}
    if E:
        rng = random.Random(seed)
        live = rng.sample(range(E), case["hit"])
        slots = [live[i % len(live)] if i < len(live) else None for i in range(rows * case["picks"])]
        for t in range(rows):                   # a row's experts are different ones, some taken more often
            mine = slots[t * case["picks"]:(t + 1) * case["picks"]]
            for i, e in enumerate(mine):
                while e is None:
                    e = live[min(int(rng.random() ** 2 * len(live)), len(live) - 1)]
                    e = None if e in mine else e
                mine[i] = e
            slots[t * case["picks"]:(t + 1) * case["picks"]] = mine
        s["expert"] = torch.tensor(slots, device="cuda").view(rows, case["picks"])
    return s


def prepare_logprobs(case, gen, seed):
    """Logits of a model that is sure of some tokens; half of the given tokens are among these."""
    rows, vocab, n, T = case["rows"], case["vocab"], case["given"], DT[case["dtype"]]
    sure = torch.randint(vocab - case["padded"], (rows, max(n, 4)), generator=gen, device="cuda")
    x = randn(gen, rows, vocab).mul_(2.5)
    x.scatter_add_(1, sure, 4 + 3 * randn(gen, rows, max(n, 4)))
    x = x.to(T)
    if case["padded"]:
        x[:, -case["padded"]:] = -math.inf
    rest = torch.randint(vocab - case["padded"], (rows, n), generator=gen, device="cuda")
    tokens = torch.where(torch.rand(rows, n, generator=gen, device="cuda") < 0.5, sure[:, :n], rest)
    gone = torch.randperm(rows, generator=gen, device="cuda")[:int(rows * case["masked"])]
    tokens[gone] = -1
    s = {"case": case, "logits": x, "tokens": tokens}
    if case["way"] == "bwd":
        s["dlogp"] = randn(gen, rows, n) / rows
        s["dentropy"] = 0.01 * randn(gen, rows) / rows
        s["stats"], s["entropy"] = torch.zeros(rows, 2, device="cuda"), torch.zeros(rows, device="cuda")
        step = max(1, (1 << 27) // vocab)       # what the forward pass left
        for a in range(0, rows, step):
            z = x[a:a + step].double()
            top = z.amax(1, keepdim=True)
            z = (z - top) / case["temperature"]
            total = z.exp().sum(1)
            p = z.exp() / total[:, None]
            s["stats"][a:a + step, 0] = top[:, 0]
            s["stats"][a:a + step, 1] = total.log()
            s["entropy"][a:a + step] = total.log() - torch.where(p > 0, p * z, 0.0).sum(1)
        s["stats"][gone] = 0
        s["entropy"][gone] = 0
    return s


def prepare_norm(case, gen, seed):
    """Gradients in the middle of training: one buffer that the tensors are parts of, every part
    starting at a multiple of 128 elements."""
    sizes = tensor_sizes(case)
    at = [0]
    for n in sizes:
        at.append(at[-1] + -(-n // 128) * 128)
    flat = torch.zeros(at[-1], dtype=DT[case["dtype"]], device="cuda")
    part = [flat[a:a + n] for a, n in zip(at, sizes)]
    for k, g in enumerate(part):
        size = math.exp(0.5 * (k % 7) - 8)            # tensors differ in size, and values within one
        g.copy_(torch.exp(randn(gen, g.numel())) * size * randn(gen, g.numel()))
    s = {"case": case, "grads": part}
    if case["way"] == "clip":
        s["out"] = torch.zeros_like(flat)
        s["outs"] = [s["out"][a:a + n] for a, n in zip(at, sizes)]
    if own:                                           # the optimizer that a program keeps
        import nvfp4_block_scaled_amax_amd as nv
        like = torch.zeros(at[-1], dtype=torch.bfloat16, device="cuda")
        s["plan"] = nv.adamw_plan([like[a:a + n] for a, n in zip(at, sizes)], state="e4m3")
    return s


# ---------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if op == "matvec":
        return packed_matvec(s) if own else plain_matvec(s)
    if op == "logprobs":
        if s["case"]["way"] == "fwd":
            return token_logprobs(s) if own else plain_logprobs(s)
        return token_logprobs_backward(s) if own else plain_logprobs_backward(s)
    return grad_norm(s) if own else plain_norm(s)


def packed_matvec(s):
    import nvfp4_block_scaled_amax_amd as nv
    return nv.packed_matvec(s["x"], s["codes"], s["scales"], s["alpha"], expert=s["expert"],
                            dtype=DT[s["case"]["out"]])


def unpack(codes, scales, alpha):
    """Packed weights of one matrix -> [n, k] in 32 bits."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], device="cuda")
    w = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), 2)
    w = w.view(codes.shape[0], -1, BLOCK) * scales.view(torch.float8_e4m3fn).float()[:, :, None]
    return w.view(codes.shape[0], -1) * alpha


def plain_matvec(s):
    case, x, T = s["case"], s["x"].float(), DT[s["case"]["out"]]
    if not case["experts"]:
        return (x @ unpack(s["codes"], s["scales"], s["alpha"]).t()).to(T)
    rows, picks = s["expert"].shape
    y = torch.zeros(rows, picks, case["n"], dtype=T, device="cuda")
    for e in range(case["experts"]):
        row, pick = torch.nonzero(s["expert"] == e, as_tuple=True)
        if row.numel():
            y[row, pick] = (x[row] @ unpack(s["codes"][e], s["scales"][e], s["alpha"][e]).t()).to(T)
    return y


def token_logprobs(s):
    import nvfp4_block_scaled_amax_amd as nv
    case = s["case"]
    logp, entropy, top_logp, top_index, stats = nv.token_logprobs(
        s["logits"], s["tokens"], top=case["top"], temperature=case["temperature"])
    out = {"logp": logp, "entropy": entropy, "stats": stats}
    if case["top"]:
        out.update(top_logp=top_logp, top_index=top_index)
    return out


def plain_logprobs(s):
    case, rows = s["case"], s["case"]["rows"]
    vocab, k, T = case["vocab"], case["top"], case["temperature"]
    parts = []
    step = max(1, (1 << 28) // vocab)
    for a in range(0, rows, step):
        x, tokens = s["logits"][a:a + step].float(), s["tokens"][a:a + step]
        live = (tokens >= 0).any(1)
        m = x.amax(1, keepdim=True)
        z = (x - m) / T
        e = torch.exp(z)
        total = e.sum(1, keepdim=True)
        log = torch.log(total)
        entropy = log[:, 0] - torch.where(e > 0, e * z, 0.0).sum(1) / total[:, 0]
        logp = torch.where(tokens >= 0, z.gather(1, tokens.clamp(min=0)) - log, 0.0)
        out = [logp, torch.where(live, entropy, 0.0),
               torch.where(live[:, None], torch.cat((m, log), 1), 0.0)]
        if k:
            # largest first, the lowest index among equals: order-preserving bits above the index
            bits = (x + 0.0).view(torch.int32).long()
            key = torch.where(bits < 0, -(1 << 31) - bits - 1, bits) * (1 << 32)
            key += vocab - 1 - torch.arange(vocab, device="cuda")
            top = vocab - 1 - (key.topk(k, dim=1).values & 0xFFFFFFFF)
            out += [torch.where(live[:, None], z.gather(1, top) - log, 0.0),
                    torch.where(live[:, None], top, -1)]
        parts.append(out)
    got = [torch.cat(p) for p in zip(*parts)]
    return dict(zip(("logp", "entropy", "stats", "top_logp", "top_index"), got))


def token_logprobs_backward(s):
    import nvfp4_block_scaled_amax_amd as nv
    return nv.token_logprobs_backward(s["logits"], s["tokens"], s["stats"], s["dlogp"],
                                      entropy=s["entropy"], dentropy=s["dentropy"],
                                      temperature=s["case"]["temperature"])


def plain_logprobs_backward(s):
    T, x, tokens = s["case"]["temperature"], s["logits"].float(), s["tokens"]
    g = torch.where(tokens >= 0, s["dlogp"], 0.0)
    live = (tokens >= 0).any(1)[:, None]
    lp = (x - s["stats"][:, :1]) / T - s["stats"][:, 1:]
    p = torch.exp(lp)
    rest = torch.where(p > 0, p * (lp + s["entropy"][:, None]), 0.0) * s["dentropy"][:, None]
    grad = -(p * g.sum(1, keepdim=True) + rest)
    grad = grad.scatter_add_(1, tokens.clamp(min=0), g) / T
    return torch.where(live, grad, 0.0).to(s["logits"].dtype)


def grad_norm(s):
    import nvfp4_block_scaled_amax_amd as nv
    norm, scale = nv.grad_norm(s["plan"], s["grads"], max_norm=1.0, eps=CLIP_EPS)
    if s["case"]["way"] == "norm":
        return {"norm": norm, "scale": scale}
    nv.clip_grads(s["plan"], s["grads"], scale, out=s["outs"])
    return {"norm": norm, "scale": scale, "out": s["out"]}


def plain_norm(s):
    total = torch.zeros(1, dtype=torch.float64, device="cuda")
    for g in s["grads"]:
        total += g.float().square().sum(dtype=torch.float64)
    norm = total.sqrt()
    scale = (1.0 / (norm + CLIP_EPS)).clamp(max=1.0).float()
    out = {"norm": norm.float(), "scale": scale}
    if s["case"]["way"] == "clip":
        for g, to in zip(s["grads"], s["outs"]):
            to.copy_(g.float() * scale)
        out["out"] = s["out"]
    return out


# ---------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matvec":
        return exact_matvec(case, s)
    if case["op"] == "logprobs":
        return exact_logprobs(case, s) if case["way"] == "fwd" else exact_logprobs_backward(case, s)
    # scaled sums of squares, tensor by tensor
    largest = max(float(g.abs().amax()) for g in s["grads"]) or 1.0
    total = sum(float(((g.double() / largest) ** 2).sum()) for g in s["grads"])
    norm = largest * math.sqrt(total)
    scale = min(1.0, 1.0 / (norm + CLIP_EPS))
    out = {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
           "scale": torch.tensor([scale], dtype=torch.float64, device="cuda")}
    if case["way"] == "clip":
        out["out"] = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for g, to in zip(s["grads"], s["outs"]):
            at = (to.data_ptr() - s["out"].data_ptr()) // to.element_size()
            out["out"][at:at + g.numel()] = g.double() * scale
    return out


def values64(codes, scales):
    """Codes and scales by their fields: sign, exponent, mantissa."""
    c = torch.stack((codes & 15, codes >> 4), 2).reshape(codes.shape[0], -1).int()
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e > 0, (1 + m / 2) * torch.exp2((e - 1).double()), m / 2)
    v = torch.where(c >= 8, -v, v)
    s = scales.int()
    e, m = (s >> 3) & 15, (s & 7).double()
    f = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m / 512)
    return v * f.repeat_interleave(BLOCK, 1)


def exact_matvec(case, s):
    x, step = s["x"].double(), max(1, (1 << 27) // case["k"])
    if not case["experts"]:
        return torch.cat([x @ values64(s["codes"][a:a + step], s["scales"][a:a + step]).t()
                          for a in range(0, case["n"], step)], 1) * s["alpha"].double()
    out = torch.zeros(case["rows"], case["picks"], case["n"], dtype=torch.float64, device="cuda")
    for e in set(s["expert"].flatten().tolist()):
        y = x @ values64(s["codes"][e], s["scales"][e]).t() * s["alpha"][e].double()
        out = torch.where((s["expert"] == e)[:, :, None], y[:, None, :], out)
    return out


def exact_logprobs(case, s):
    out = {"logp": [], "entropy": [], "stats": []}
    if case["top"]:
        out.update(top_logp=[], top_index=[])
    step = max(1, (1 << 26) // case["vocab"])
    for a in range(0, case["rows"], step):
        x, tokens = s["logits"][a:a + step].double(), s["tokens"][a:a + step]
        lp = torch.log_softmax(x / case["temperature"], 1)
        gone = ~(tokens >= 0).any(1)
        given = lp.gather(1, tokens.clamp(min=0))
        given[tokens < 0] = 0
        h = -(lp.exp() * lp.clamp(min=-1e300)).sum(1)
        m = x.amax(1)
        stats = torch.stack((m, torch.logsumexp((x - m[:, None]) / case["temperature"], 1)), 1)
        row = {"logp": given, "entropy": h, "stats": stats}
        if case["top"]:
            index = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["top"]]
            row["top_logp"], row["top_index"] = lp.gather(1, index), index
        for k, v in row.items():
            v[gone] = -1 if k == "top_index" else 0
            out[k].append(v)
    return {k: torch.cat(v) for k, v in out.items()}


def exact_logprobs_backward(case, s):
    """The chain through log_softmax, from the logits alone."""
    parts, T = [], case["temperature"]
    big = case["rows"] * case["vocab"] >= 1 << 28
    step = max(1, (1 << 26) // case["vocab"])
    for a in range(0, case["rows"], step):
        tokens = s["tokens"][a:a + step]
        lp = torch.log_softmax(s["logits"][a:a + step].double() / T, 1)
        p = lp.exp()
        low = lp.clamp(min=-1e300)
        h = -(p * low).sum(1, keepdim=True)
        up = -(low + h) * p * s["dentropy"][a:a + step, None].double()      # of the entropy
        d = s["dlogp"][a:a + step].double() * (tokens >= 0)
        up -= p * d.sum(1, keepdim=True)
        up.scatter_add_(1, tokens.clamp(min=0), d)
        up *= (tokens >= 0).any(1, keepdim=True) / T
        parts.append(up.float() if big else up)
    return torch.cat(parts)
