"""Measured cases of the matrix operators: the Newton-Schulz orthogonalisation, the Muon
step built on it, the 4-bit microscaled copy of a weight matrix, and the product of two
such copies.

`run` computes an operator in its plain form (elementary torch operations in 32 bits) or,
where `own` is true, through mixed_precision_zero_amd.matrix.
"""
import math

import torch

own = False

DEV = "cuda"
NS_COEF = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
NS_EPS = 1e-7
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# What the optimizer cases run with: the library's defaults and the step size of its
# workloads, a loss scale that stays where it is, weights of the workloads' spread.
LR = 6e-4
MOMENTUM = 0.95
DECAY = 0.01
CLIP = 1.0
LOSS_SCALE = 1024.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------

def listed():
    return [
        # the projections of 64 small heads, orthogonalised one by one: launch latency
        dict(name="orth 64 x 64x64", op="orth", count=64, rows=64, cols=64, src="f32", dst="bf16"),
        # a narrow adapter pair's odd-sized factor: nothing is a multiple of a tile
        dict(name="orth 387x1001", op="orth", count=1, rows=387, cols=1001, src="bf16", dst="bf16"),
        # Pythia-410M MLP input weights of eight layers (4096 out, 1024 in): tall
        dict(name="orth 8 x 4096x1024", op="orth", count=8, rows=4096, cols=1024, src="f16", dst="f16"),
        # GPT-NeoX-20B attention output weight (hidden 6144)
        dict(name="orth 6144x6144", op="orth", count=1, rows=6144, cols=6144, src="f32", dst="bf16"),
        # one step over four small square weights: launch latency of the whole step
        dict(name="muon 4 x 256x256", op="muon", count=4, rows=256, cols=256, dtype="f16",
             nesterov=True, scale="rms"),
        # Pythia-410M: MLP weights of four layers
        dict(name="muon 4 x 1024x4096", op="muon", count=4, rows=1024, cols=4096, dtype="f16",
             nesterov=True, scale="rms"),
        # GPT-NeoX-20B MLP input weight (24576 out, 6144 in), bf16 gradients, plain momentum
        dict(name="muon 24576x6144", op="muon", count=1, rows=24576, cols=6144, dtype="bf16",
             nesterov=False, scale="rms"),
        # the 4-bit copy a rank sends after its step and the half weights its peers read from
        # it: an odd-sized weight, and the GPT-NeoX-20B MLP weight with its transpose too
        dict(name="copy 1000x1037", op="copy", rows=1000, cols=1037, src="f32", dst="f16",
             both=False),
        dict(name="copy 24576x6144 both", op="copy", rows=24576, cols=6144, src="f32", dst="bf16",
             both=True),
        # one token through the GPT-NeoX-20B MLP input weight
        dict(name="product 1x24576x6144", op="product", m=1, n=24576, k=6144, src="bf16",
             dst="bf16"),
        # a short ragged batch of tokens through a Pythia-410M MLP weight, sums kept
        dict(name="product 333x4096x1024", op="product", m=333, n=4096, k=1024, src="f16",
             dst="f32"),
        # a training batch through the GPT-NeoX-20B MLP input weight
        dict(name="product 8192x24576x6144", op="product", m=8192, n=24576, k=6144, src="bf16",
             dst="bf16"),
    ]


def _size(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:                 # half of the sizes round, half as they fall
        step = 64 if n >= 256 else 8
        n = max(lo, n // step * step)
    return n


def draw(rng):
    op = rng.choice(("orth", "muon", "copy", "product"))
    if op == "orth":
        rows, cols = _size(rng, 32, 6144), _size(rng, 32, 6144)
        most = max(1, min(64, (1 << 25) // (rows * cols)))
        return dict(op=op, count=_size(rng, 1, most + 1) if most > 1 else 1, rows=rows, cols=cols,
                    src=rng.choice(("f32", "f16", "bf16")), dst=rng.choice(("f16", "bf16")))
    if op == "muon":
        rows, cols = _size(rng, 64, 8192), _size(rng, 64, 6144)
        most = max(1, min(16, (1 << 25) // (rows * cols)))
        return dict(op=op, count=rng.randint(1, most), rows=rows, cols=cols,
                    dtype=rng.choice(("f16", "bf16")), nesterov=rng.random() < 0.7, scale="rms")
    if op == "copy":
        return dict(op=op, rows=_size(rng, 64, 16384), cols=_size(rng, 64, 8192),
                    src=rng.choice(("f32", "f16", "bf16")), dst=rng.choice(("f16", "bf16")),
                    both=rng.random() < 0.5)
    return dict(op=op, m=_size(rng, 1, 8192), n=_size(rng, 64, 24576), k=_size(rng, 64, 6144),
                src=rng.choice(("f16", "bf16")), dst=rng.choice(("f32", "f16", "bf16")))


def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}
    if case["op"] in ("orth", "muon"):
        m, n = sorted((case["rows"], case["cols"]))
        # both symmetric products need one half only
        flops = case["count"] * NS_STEPS * (m * m * n + m * m * m + 2 * m * m * n)
        numel = case["count"] * m * n
        if case["op"] == "orth":
            return {"bytes": numel * (size[case["src"]] + size[case["dst"]]), "flops": flops}
        # gradient, momentum and master read, momentum, master and half written
        return {"bytes": numel * (2 + 4 + 4 + 4 + 4 + 2), "flops": flops}
    if case["op"] == "copy":
        numel, times = case["rows"] * case["cols"], 2 if case["both"] else 1
        # the matrix is read once; each copy is written, read back and written out
        return {"bytes": numel * (size[case["src"]] + times * (2 * 17 / 32 + size[case["dst"]])),
                "flops": 0}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": m * k * size[case["src"]] + n * k * 17 / 32 + m * n * size[case["dst"]],
            "flops": 2 * m * n * k}


# ----------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------

def _momentum_like(gen, rows, cols, sigma):
    """A few strong directions over noise, as a gradient or its running average has."""
    r = min(8, rows, cols)
    u = torch.randn(rows, r, generator=gen, device=DEV)
    v = torch.randn(r, cols, generator=gen, device=DEV)
    return (u @ v * (0.5 / math.sqrt(r)) + torch.randn(rows, cols, generator=gen, device=DEV)) * sigma


def _pack(x):
    """(codes, scales) of x's rows, two elements a byte, rows padded to 128 elements."""
    scale, q = _mx_parts(x)
    rows, cols = x.shape
    wide = -(-cols // 128) * 128
    codes = torch.zeros(rows, wide, dtype=torch.uint8, device=DEV)
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    codes[:, :cols] = (code + torch.where(q < 0, 8, 0).to(torch.uint8))[:, :cols]
    scales = torch.zeros(rows, wide // 32, dtype=torch.uint8, device=DEV)
    scales[:, :scale.shape[1]] = (scale + 127).to(torch.uint8)
    pairs = codes.view(rows, wide // 2, 2)
    return (pairs[:, :, 0] | pairs[:, :, 1] << 4).contiguous(), scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    if op == "orth":
        x = torch.stack([_momentum_like(gen, case["rows"], case["cols"], 1e-3)
                         for _ in range(case["count"])])
        return {"case": case, "x": x.to(DTYPES[case["src"]])}
    if op == "muon":
        dt, shape = DTYPES[case["dtype"]], (case["rows"], case["cols"])
        mats = []
        for i in range(case["count"]):
            master = torch.randn(shape, generator=gen, device=DEV) * 0.02
            mats.append({"grad": (_momentum_like(gen, *shape, 1e-4) * LOSS_SCALE).to(dt),
                         "half": master.to(dt), "master": master,
                         "momentum": _momentum_like(gen, *shape, 5e-4), "decay": i % 4 != 3})
        state = {"case": case, "mats": mats}
        if own:
            import mixed_precision_zero_amd as Z
            from mixed_precision_zero_amd import matrix as M
            cfg = Z.neox_zero1_default_config(
                beta1=MOMENTUM, weight_decay=DECAY, clip_norm=CLIP, init_scale=LOSS_SCALE,
                scaler_mode=Z.NEOX_SCALER_STATIC,
                dtype=Z.NEOX_F16 if dt == torch.float16 else Z.NEOX_BF16)
            mcfg = M.neox_muon_default_config(
                nesterov=int(case["nesterov"]),
                scale_mode=M.NEOX_MUON_SCALE_RMS if case["scale"] == "rms"
                else M.NEOX_MUON_SCALE_SHAPE)
            state["opt"] = M.Muon(cfg, [M.muon_matrix(**t) for t in mats], mcfg)
        return state
    if op == "copy":
        x = torch.randn(case["rows"], case["cols"], generator=gen, device=DEV) * 0.02
        return {"case": case, "x": x.to(DTYPES[case["src"]])}
    w = torch.randn(case["n"], case["k"], generator=gen, device=DEV) * 0.02
    x = torch.randn(case["m"], case["k"], generator=gen, device=DEV)
    loud = torch.rand(case["k"], generator=gen, device=DEV) < 0.01   # a few strong channels
    x = torch.where(loud, x * 12, x)
    codes, scales = _pack(w)
    return {"case": case, "x": x.to(DTYPES[case["src"]]), "codes": codes, "scales": scales}


# ----------------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------------

def _newton_schulz(g):
    x = g.float()
    if x.shape[-2] > x.shape[-1]:
        return _newton_schulz(x.transpose(-1, -2).contiguous()).transpose(-1, -2)
    a, b, c = NS_COEF
    norm = x.double().square().sum((-2, -1), keepdim=True).sqrt().float()
    x = x / (norm + NS_EPS)
    for _ in range(NS_STEPS):
        p = torch.matmul(x, x.transpose(-1, -2).contiguous())
        x = a * x + torch.matmul(b * p + c * torch.matmul(p, p), x)
    return x


def _muon(case, mats):
    sq, unscaled = None, []
    for t in mats:
        g = t["grad"].float() * (1.0 / LOSS_SCALE)
        unscaled.append(g)
        s = g.double().square().sum()
        sq = s if sq is None else sq + s
    norm = sq.sqrt()
    applied = torch.isfinite(norm)
    coef = torch.where(norm > CLIP, CLIP / norm, torch.ones_like(norm)).float()
    scale = 0.2 * math.sqrt(max(case["rows"], case["cols"])) if case["scale"] == "rms" \
        else math.sqrt(max(1.0, case["rows"] / case["cols"]))
    outs = []
    for t, g in zip(mats, unscaled):
        g = g * coef
        m = MOMENTUM * t["momentum"] + g
        o = _newton_schulz(g + MOMENTUM * m if case["nesterov"] else m) * scale
        w = t["master"] - LR * (o + (DECAY if t["decay"] else 0.0) * t["master"])
        t["momentum"].copy_(torch.where(applied, m, t["momentum"]))
        t["master"].copy_(torch.where(applied, w, t["master"]))
        t["half"].copy_(torch.where(applied, w.to(t["half"].dtype), t["half"]))
        outs.append((t["master"], t["momentum"], t["half"]))
    return outs


def _mx_parts(x):
    """The block exponents (rows, blocks) and the elements rounded to E2M1, unscaled, of x's
    rows padded to whole blocks of 32."""
    rows, cols = x.shape
    x = x.float()
    if cols % 32:
        x = torch.cat([x, x.new_zeros(rows, -cols % 32)], 1)
    x = x.view(rows, -1, 32)
    e = torch.frexp(x.abs().amax(-1)).exponent - 3           # floor(log2 amax) - 2
    e = torch.where(x.abs().amax(-1) > 0, e.clamp(min=-127), -127)
    v = torch.ldexp(x, -e.unsqueeze(-1))
    a = v.abs()
    r = torch.where(a < 2, torch.round(a * 2) / 2,
                    torch.where(a < 4, torch.round(a), (torch.round(a / 2) * 2).clamp(max=6)))
    return e, torch.where(v < 0, -r, r).reshape(rows, -1)


def _mx_values(x):
    e, q = _mx_parts(x)
    v = torch.ldexp(q.view(q.shape[0], -1, 32), e.unsqueeze(-1))
    return v.reshape(q.shape)[:, :x.shape[1]]


def _unpack(codes, scales, cols):
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    both = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1)
    v = lut[both.long()].view(codes.shape[0], -1, 32)
    return torch.ldexp(v, scales.int().unsqueeze(-1) - 127).reshape(codes.shape[0], -1)[:, :cols]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(state, case, op)
    if op == "orth":
        return _newton_schulz(state["x"]).to(DTYPES[case["dst"]])
    if op == "muon":
        return _muon(case, state["mats"])
    if op == "copy":
        dt, x = DTYPES[case["dst"]], state["x"]
        out = [_mx_values(x).to(dt)]
        if case["both"]:
            out.append(_mx_values(x.t().contiguous()).to(dt))
        return out
    w = _unpack(state["codes"], state["scales"], case["k"])
    return torch.matmul(_mx_values(state["x"]), w.t()).to(DTYPES[case["dst"]])


def _run_own(state, case, op):
    from mixed_precision_zero_amd import matrix as M
    if op == "orth":
        return M.orthogonalize(state["x"], dtype=DTYPES[case["dst"]])
    if op == "muon":
        state["opt"].step(LR)
        return [(t["master"], t["momentum"], t["half"]) for t in state["mats"]]
    if op == "copy":
        dt, x = DTYPES[case["dst"]], state["x"]
        out = [M.mxfp4_dequantize(M.mxfp4_quantize(x), dt)]
        if case["both"]:
            out.append(M.mxfp4_dequantize(M.mxfp4_quantize(x, transpose=True), dt))
        return out
    w = M.MXFP4(state["codes"], state["scales"], case["n"], case["k"])
    return M.mxfp4_product(M.mxfp4_quantize(state["x"]), w, DTYPES[case["dst"]])


# ----------------------------------------------------------------------------------------
# 64 bits, from the definitions
# ----------------------------------------------------------------------------------------

def _exact_orth(g):
    """The same polynomial applied from the other side, X (a I + b X'X + c (X'X)^2), on the
    narrow side's Gram matrix."""
    g = g.double()
    if g.shape[0] < g.shape[1]:
        return _exact_orth(g.t()).t()
    a, b, c = NS_COEF
    x = g / (torch.linalg.vector_norm(g) + NS_EPS)
    eye = torch.eye(x.shape[1], dtype=torch.float64, device=x.device)
    for _ in range(NS_STEPS):
        s = x.t().contiguous() @ x
        x = x @ (a * eye + s @ (b * eye + c * s))
    return x


def _exact_mx(x):
    """Every element to the nearest of the fifteen values, by distance, ties to the even code."""
    x = x.double()
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % 32)).view(rows, -1, 32)
    top = x.abs().amax(-1, keepdim=True)
    expo = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    # log2 in 64 bits may round up to a power of two that the block does not reach
    expo = torch.where(torch.exp2(expo) > top, expo - 1, expo)
    scale = torch.exp2((expo - 2).clamp(min=-127))
    mag = (x.abs() / scale).clamp(max=6.0)
    best, far = torch.zeros_like(mag), mag.clone()
    for code in (2, 4, 6, 1, 3, 5, 7):                # even codes first: they keep ties
        d = (mag - E2M1[code]).abs()
        nearer = d < far
        best, far = torch.where(nearer, torch.full_like(best, E2M1[code]), best), torch.where(nearer, d, far)
    return (torch.sign(x) * best * scale).reshape(rows, -1)[:, :cols]


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "orth":
        return torch.stack([_exact_orth(x) for x in state["x"]])
    if op == "muon":
        grads = [t["grad"].double() / LOSS_SCALE for t in state["mats"]]
        norm = math.sqrt(sum(float((g * g).sum()) for g in grads))
        coef = CLIP / norm if norm > CLIP else 1.0
        scale = 0.2 * math.sqrt(max(case["rows"], case["cols"])) if case["scale"] == "rms" \
            else math.sqrt(max(1.0, case["rows"] / case["cols"]))
        out = []
        for t, g in zip(state["mats"], grads):
            g = g * coef
            m = t["momentum"].double() * MOMENTUM + g
            w = t["master"].double()
            step = scale * _exact_orth(m * MOMENTUM + g if case["nesterov"] else m)
            w = w - LR * (step + (DECAY * w if t["decay"] else 0.0))
            out.append((w, m, w))
        return out
    if op == "copy":
        out = [_exact_mx(state["x"])]
        if case["both"]:
            out.append(_exact_mx(state["x"].t()))
        return out
    codes, scales = state["codes"].long(), state["scales"].double()
    w = torch.empty(case["n"], codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
    for half, nib in enumerate((codes % 16, codes // 16)):
        mag, ex = nib % 2, nib // 2 % 4               # mantissa bit, exponent field
        v = torch.where(ex == 0, mag * 0.5, (1 + mag * 0.5) * torch.exp2(ex.double() - 1))
        w[:, half::2] = torch.where(nib >= 8, -v, v)
    w *= torch.exp2(scales - 127).repeat_interleave(32, 1)
    return _exact_mx(state["x"]) @ w[:, :case["k"]].t()
