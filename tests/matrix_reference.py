"""Plain 64-bit forms of the matrix operators for the tests: the Newton-Schulz polynomial
(and the same with the kernels' roundings, to size tolerances), the Muon update, and MXFP4
element by element.  torch on the CPU; nothing here uses the library."""
import math

import torch

COEF = [(3.4445, -4.7750, 2.0315)] * 5
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def newton_schulz(g, coef=COEF, eps=1e-7):
    """64 bits; g: (rows, cols)."""
    x = g.double().cpu()
    if x.shape[0] > x.shape[1]:
        return newton_schulz(x.t(), coef, eps).t()
    x = x / (torch.linalg.vector_norm(x) + eps)
    for a, b, c in coef:
        p = x @ x.t()
        x = a * x + (b * p + c * (p @ p)) @ x
    return x


def newton_schulz_rounded(g, coef=COEF, eps=1e-7):
    """The same with every rounding the kernels make (FP16 product operands, the iterate as two
    FP16 numbers, diagonals apart, two steps at a time where the kernels take them so) and
    64-bit sums: its distance from newton_schulz() is what those roundings cost on this input."""
    x = g.double().cpu()
    m, n = x.shape
    if m > n:
        return newton_schulz_rounded(x.t(), coef, eps).t()
    half = lambda t: t.to(torch.float16).double()  # noqa: E731

    def apart(p):
        d = torch.diag(p).clone()
        return d, half(p - torch.diag(d))

    def times(d, o, e, p):
        return o @ p + d[:, None] * p + o * e[None, :] + torch.diag(d * e)

    def poly(d, o, abc):
        a, b, c = abc
        return apart(a * torch.eye(m, dtype=torch.float64) + b * (o + torch.diag(d)) + c * times(d, o, d, o))

    s = 2.0 ** math.floor((math.floor(math.log2(n)) + 1) / 2)
    x = x / (torch.linalg.vector_norm(x) + eps) * s
    k = 0
    while k < len(coef):
        hi = half(x)
        x = hi + half((x - hi) * 2048) / 2048
        gram = apart(hi @ hi.t() / s ** 2)
        p = poly(*gram, coef[k])
        if m > 512 and n >= 2 * m and k + 1 < len(coef):
            gram = apart(times(*apart(times(*p, *gram)), *p))
            p = apart(times(*poly(*gram, coef[k + 1]), *p))
            k += 1
        x = p[0][:, None] * x + p[1] @ hi
        k += 1
    return x / s


def rms(t):
    return float(t.double().square().mean().sqrt())


def orth_bounds(g, dtype, coef=COEF, eps=1e-7):
    """(exact result, bound on the rms of the error, bound on any element's error).

    The roundings are pseudo-random, so another order of the FP32 sums flips some of them and
    gives an error of the same size but of other signs: three times the model's rms (and, for
    single elements, three times its largest).  Besides: half a step of the output type per
    element, and FP32 sums, 2^-24 a term along both products of five steps, far below."""
    want = newton_schulz(g, coef, eps)
    err = newton_schulz_rounded(g, coef, eps) - want
    u = torch.finfo(dtype).eps / 2
    top, n = float(want.abs().max()), max(g.shape)
    f32 = 5 * 2 * math.sqrt(n) * 2.0 ** -24
    return (want, 3 * rms(err) + u * rms(want) + f32 * rms(want) + 1e-30,
            3 * float(err.abs().max()) + u * top + 8 * f32 * top + 2.0 ** -24)


def check_orth(got, g, scale=1.0, coef=COEF, eps=1e-7):
    want, r, m = orth_bounds(g, got.dtype, coef, eps)
    d = got.double().cpu() / scale - want
    assert torch.isfinite(d).all()
    assert rms(d) <= r, (rms(d), r)
    assert float(d.abs().max()) <= m, (float(d.abs().max()), m)


# ----------------------------------------------------------------------------------------
# MXFP4
# ----------------------------------------------------------------------------------------

def mx_quantize(x):
    """-> (codes (R, K/2) uint8, scales (R, K/32) uint8) of x (R, C), in 64 bits."""
    x = x.detach().cpu().double()
    rows, cols = x.shape
    k = -(-cols // 128) * 128
    v = torch.zeros(rows, k, dtype=torch.float64)
    v[:, :cols] = x
    v = v.view(rows, k // 32, 32)
    bad = ~torch.isfinite(v).all(-1)
    top = torch.where(torch.isfinite(v), v, torch.zeros_like(v)).abs().amax(-1)
    e = torch.frexp(top).exponent.double() - 1 - 2               # floor(log2 top) - 2
    e = torch.where(top > 0, e.clamp(min=-127), torch.full_like(e, -127))
    mag = torch.where(bad[..., None], torch.zeros_like(v), v.abs() * torch.exp2(-e)[..., None])
    # nearest value, ties to the even code: midpoints belong to the even neighbour
    code = torch.zeros_like(mag, dtype=torch.int64)
    for c in range(7):
        mid = (E2M1[c] + E2M1[c + 1]) / 2
        code += ((mag > mid) | ((mag == mid) & (c % 2 == 1))).long()
    neg = torch.signbit(torch.where(bad[..., None], torch.zeros_like(v), v))
    code = (code + 8 * neg.long()).view(rows, k)
    packed = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    scale = torch.where(bad, torch.full_like(e, 255.0), e + 127).to(torch.uint8)
    return packed, scale


def mx_values(codes, scales, cols):
    codes, scales = codes.cpu().long(), scales.cpu().double()
    nib = torch.stack([codes % 16, codes // 16], -1).view(codes.shape[0], -1)
    table = torch.tensor(list(E2M1) + [-v for v in E2M1], dtype=torch.float64)
    v = table[nib].view(codes.shape[0], -1, 32)
    f = torch.where(scales == 255, torch.full_like(scales, math.nan), torch.exp2(scales - 127))
    return (v * f[..., None]).reshape(codes.shape[0], -1)[:, :cols]


# ----------------------------------------------------------------------------------------
# Muon
# ----------------------------------------------------------------------------------------

def muon_scale(rows, cols, mode):
    return 0.2 * math.sqrt(max(rows, cols)) if mode == "rms" else math.sqrt(max(1.0, rows / cols))
