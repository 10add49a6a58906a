"""Plain forms of the linear layer's operators in 64 bits, on the CPU, and the errors their
FP32 evaluation may have."""
import math

import numpy as np
import torch

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = 2.0 ** -24                       # half a step of FP32
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def philox(counter, key):
    """Philox-4x32-10 of one counter (four words) and key (two), in Python's integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def draws(seed, offset, rows, cols, first_row=0):
    """The 16 random bits of each element."""
    u = np.uint64
    wide = -(-cols // 8)
    m = u(0xFFFFFFFF)
    c = [np.broadcast_to(np.arange(wide, dtype=u), (rows, wide)),
         np.broadcast_to(np.arange(first_row, first_row + rows, dtype=u)[:, None], (rows, wide)),
         np.full((rows, wide), offset & 0xFFFFFFFF, dtype=u), np.full((rows, wide), offset >> 32, dtype=u)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = u(0xD2511F53) * c[0], u(0xCD9E8D57) * c[2]
        c = [(b >> u(32)) ^ c[1] ^ u(k0), b & m, (a >> u(32)) ^ c[3] ^ u(k1), a & m]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = np.stack(c, -1)
    both = np.stack([words & u(0xFFFF), words >> u(16)], -1)
    return torch.from_numpy(both.reshape(rows, wide * 8)[:, :cols].astype(np.int64))


def limit_of(p):
    return round(p * 65536)          # ties to even


def keep(drop, rows, cols):
    """(what each element is multiplied by if it is kept, whether it is): drop = (p, seed, offset)."""
    if drop is None or limit_of(drop[0]) == 0:
        return 1.0, torch.ones(rows, cols, dtype=torch.bool)
    t = limit_of(drop[0])
    scale = 0.0 if t == 65536 else float(np.float32(65536 / (65536 - t)))
    return scale, draws(drop[1], drop[2], rows, cols) >= t


def dropped(v, drop):
    scale, k = keep(drop, *v.shape)
    return torch.where(k, v * scale, torch.zeros((), dtype=v.dtype))


def act(name, v):
    if name == "none":
        return v
    y = {"relu": lambda: torch.clamp(v, min=0),
         "gelu": lambda: v * 0.5 * torch.special.erfc(v * -math.sqrt(0.5)),
         "gelu_tanh": lambda: v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)),
         "silu": lambda: v * torch.sigmoid(v)}[name]()
    return torch.where(v == -math.inf, torch.zeros_like(v), y)


def slope(name, v):
    if name == "none":
        return torch.ones_like(v)
    if name == "relu":
        return torch.where(v > 0, 1.0, torch.where(v <= 0, 0.0, v))
    if name == "gelu":
        y = 0.5 * torch.special.erfc(v * -math.sqrt(0.5)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    elif name == "gelu_tanh":
        s = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
        y = s + v * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v * v)
    else:
        s = torch.sigmoid(v)
        y = s + v * s * (1 - s)
    return torch.where(v == -math.inf, torch.zeros_like(v), torch.where(v == math.inf, torch.ones_like(v), y))


def act_error(name, v):
    """How far FP32's act of an FP32 v may be off: its own roundings (at most 12 of half a step:
    the polynomial's last ones, exp2, the reciprocal, products), and those of the exponent's
    argument, three of them relative to the argument."""
    arg = {"none": 0 * v, "relu": 0 * v, "gelu": 0.5 * v * v,
           "gelu_tanh": 1.6 * v.abs() * (1 + 0.045 * v * v), "silu": v.abs()}[name]
    if name in ("none", "relu"):
        return 0 * v
    # behind these the value is taken as its limit
    return (act(name, v).abs() * U * (12 + 4 * arg)).nan_to_num(0.0) + 1e-35


def slope_error(name, v):
    """The same of a slope: a part of at most 1 and v times a bell, each with up to 12 roundings,
    and the bell's exponential with those of its argument."""
    if name in ("none", "relu"):
        return 0 * v
    w = v.clamp(-16, 16)
    if name == "gelu":
        arg, bell = 0.5 * w * w, torch.exp(-0.5 * w * w) / math.sqrt(2 * math.pi)
    elif name == "gelu_tanh":
        s = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (w + 0.044715 * w ** 3))
        arg, bell = 1.6 * w.abs() * (1 + 0.045 * w * w), s * (1 - s) * 1.6 * (1 + 0.135 * w * w)
    else:
        s = torch.sigmoid(w)
        arg, bell = w.abs(), s * (1 - s)
    return U * (12 + (1 + w.abs()) * bell * (12 + 4 * arg)) + 1e-35


def forward(x, w, bias=None, act_name="none", drop=None, residual=None):
    """(y, pre, bound on FP32's error of y before its last rounding, the same of pre)."""
    x, w = x.double().cpu(), w.double().cpu()
    v = x @ w.t()
    # k products, exact in FP32, k sums, one more for the bias
    size = x.abs() @ w.abs().t()
    if bias is not None:
        v = v + bias.double().cpu()
        size = size + bias.double().cpu().abs()
    ev = size * U * (x.shape[1] + 2)
    y = act(act_name, v)
    scale, k = keep(drop, *v.shape)
    y = torch.where(k, y * scale, torch.zeros((), dtype=y.dtype))
    # no act is steeper than 1.13
    ey = torch.where(k, (1.13 * ev + act_error(act_name, v)) * scale + y.abs() * U, torch.zeros((), dtype=y.dtype))
    if residual is not None:
        y = y + residual.double().cpu()
        ey = ey + y.abs() * U
    return y, v, ey, ev


def backward(dy, x=None, w=None, pre=None, act_name="none", drop=None):
    """d, its bound after rounding to half, and (dx, dw, dbias) with their bounds."""
    half = dy.dtype
    g = dy.double().cpu()
    scale, k = keep(drop, *g.shape)
    s = slope(act_name, pre.double().cpu()) if act_name != "none" else torch.ones_like(g)
    es = slope_error(act_name, pre.double().cpu()) if act_name != "none" else 0 * g
    d = torch.where(k, g * s * scale, torch.zeros((), dtype=g.dtype))
    e32 = torch.where(k, g.abs() * scale * es, torch.zeros((), dtype=g.dtype)) + 2 * U * d.abs()
    made = act_name != "none" or (drop is not None and limit_of(drop[0]) > 0)
    tiny = torch.finfo(half).smallest_normal * half_step(half)       # below the normal range
    e16 = e32 + ((half_step(half) * (d.abs() + e32) + tiny) if made else 0.0)
    if not made:
        e32 = 0 * e32
    out = {}
    if w is not None:
        w = w.double().cpu()
        out["dx"] = d @ w, e16 @ w.abs() + U * (d.shape[1] + 1) * ((d.abs() + e16) @ w.abs())
    if x is not None:
        x = x.double().cpu()
        out["dw"] = d.t() @ x, e16.t() @ x.abs() + U * (d.shape[0] + 1) * ((d.abs() + e16).t() @ x.abs())
    out["dbias"] = d.sum(0), e32.sum(0) + U * (d.shape[0] + 1) * (d.abs() + e32).sum(0)
    return d, e16, out


def close(got, want, bound, what=""):
    """got, in its type, within the bound and its own rounding of want.  Infinities and NaN
    have to be the same."""
    dtype = got.dtype
    g, want = got.double().cpu(), want.double()
    ok = torch.isfinite(want) & (want.abs() + bound < torch.finfo(dtype).max)
    same = torch.where(torch.isnan(want), torch.isnan(g), g == want)
    odd = ~torch.isfinite(want) & ~same
    assert not odd.any(), f"{what}: {int(odd.sum())} values that should be inf or NaN differ"
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    room = bound + half_step(dtype) * (want.abs() + bound) + tiny
    bad = ok & ~((g - want).abs() <= room)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((g - want).abs() / room)[bad].max()):.3g} times the bound, first at "
                           f"{bad.nonzero()[0].tolist()}: {g[bad][0]} for {want[bad][0]}")
