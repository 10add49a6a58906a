"""The linear layer's operators on the GPU where calls are unusual: operands that are one array,
no tokens, gradients at the top of their type's range behind dropout; and
what a tolerance would hide: bits that nothing changes, gradients element by element."""
import math

import pytest

torch = pytest.importorskip("torch")

import linear_reference as R  # noqa: E402
from mixed_precision_zero_amd import linear as L  # noqa: E402
from test_gpu_linear import BF16, F16, F32, HALVES, drops, every_half, inside, ints, rand, same_bits  # noqa: E402

pytestmark = pytest.mark.gpu


@HALVES
@pytest.mark.parametrize("side,before,extra", [(64, 0, 0), (64, 3, 5), (33, 0, 0), (300, 1, 7)])
def test_operands_that_are_one_array(side, before, extra, half):
    """dy, x and w by one address: the bits of three arrays of the same values, in whole numbers."""
    t = ints((side, side), 1, half)
    a = inside(t, before, extra)[1]
    v = t.double()
    y, _ = L.linear(a, a)
    assert same_bits(y, (v @ v.t().contiguous() + 0.0).to(half))
    dx, dw, db = L.linear_backward(a, a, a, dbias=True)
    assert same_bits(dx, (v @ v + 0.0).to(half))
    assert same_bits(dw, (v.t().contiguous() @ v + 0.0).to(half))
    assert same_bits(db, (v.sum(0) + 0.0).to(half))


@HALVES
def test_no_tokens_leave_accumulated_gradients_as_they_were(half):
    """To the bit: negative zeros, infinities and NaN with their bits among them."""
    n, k = 40, 56
    odd = torch.tensor([-0.0, 0.0, 1.0, -1.0], dtype=half, device="cuda:0").view(torch.int16)
    odd = torch.cat([odd, torch.tensor([0x7F81, -0x7F, 0x7C01, 0x7F80], dtype=torch.int16, device="cuda:0")])
    dw, db = odd.repeat(n * k // 8).view(half).view(n, k), odd.repeat(n // 8).view(half)
    was_w, was_b = dw.clone(), db.clone()
    dy, x, pre = (torch.empty(0, c, dtype=half, device="cuda:0") for c in (n, k, n))
    for act in ("none", "gelu"):
        L.linear_backward(dy, x, None, pre, act, dx=False, dw=dw, dbias=db, accumulate=True)
        assert same_bits(dw, was_w) and same_bits(db, was_b)
    L.dropout_backward(dy, L.Dropout(0.5, 1), dx=False, dbias=db, accumulate=True)
    assert same_bits(db, was_b)


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("p", [0.25, 0.5, 0.9])
@pytest.mark.parametrize("m,n,k", [(5, 96, 40), (96, 72, 200), (300, 96, 264)])
def test_dropout_does_not_overflow_gradients(m, n, k, p, act):
    """dy of up to 60000 in FP16, which dropout's factor of 1.3 to 10 takes beyond the type's range:
    dx, dw and dbias are finite, and so are the results (slopes are 1 where an act is)."""
    half = torch.float16
    dy = (rand((m, n), 1, torch.float32).sign() * 60000).to(half)
    x, w = rand((m, k), 2, half, 2.0 ** -12), rand((n, k), 3, half, 2.0 ** -12)
    pre = torch.full((m, n), 20.0, dtype=half, device="cuda:0")
    drop, ref = drops(p)
    got = dict(zip(("dx", "dw", "dbias"), L.linear_backward(dy, x, w, pre, act, drop, dbias=True)))
    want = R.backward(dy, x, w, pre, act, ref)[2]
    for name in ("dx", "dw"):
        assert float(want[name][0].abs().max()) < 60000 and bool(torch.isfinite(got[name]).all()), name
        R.close(got[name], *want[name], what=name)
    R.close(got["dbias"], *want["dbias"], what="dbias")


@HALVES
@pytest.mark.parametrize("p", [0.25, 0.3, 0.9])
@pytest.mark.parametrize("m,n,k", [(1, 50, 70), (37, 129, 260), (300, 264, 136), (333, 64, 4096), (64, 64, 16384)])
def test_dropout_without_act_rounds_no_operand(m, n, k, p, half):
    """Whole numbers, so that the sums of what is kept are exact: the results are those times
    dropout's factor, off by FP32's roundings of the product and of what it is added to, and by their
    own to half."""
    dy, x, w = ints((m, n), 1, half), ints((m, k), 2, half), ints((n, k), 3, half)
    old_w, old_b = ints((n, k), 4, half, 50), ints((n,), 5, half, 50)
    drop, ref = drops(p)
    scale, kept = R.keep(ref, m, n)
    d = torch.where(kept, dy.double().cpu(), 0.0)
    dx, dw, db = L.linear_backward(dy, x, w, dropout=drop, dbias=True)
    sums = d @ w.double().cpu(), d.t() @ x.double().cpu(), d.sum(0)
    assert all(float(v.abs().max()) < 2 ** 24 for v in sums)
    for got, v, name in zip((dx, dw, db), sums, ("dx", "dw", "dbias")):
        # (dbias adds up m products with the factor, each with a rounding)
        err = R.U * scale * (v.abs() if name != "dbias" else (m + 1) * d.abs().sum(0))
        R.close(got, v * scale, err, name)
    L.linear_backward(dy, x, None, dropout=drop, dx=False, dw=old_w, dbias=old_b, accumulate=True)
    total = sums[1] * scale + ints((n, k), 4, half, 50).double().cpu()
    R.close(old_w, total, R.U * (scale * sums[1].abs() + total.abs()), "dw, added")
    total = sums[2] * scale + ints((n,), 5, half, 50).double().cpu()
    R.close(old_b, total, R.U * (scale * (m + 1) * d.abs().sum(0) + total.abs()), "dbias, added")


@pytest.mark.parametrize("dtype", [F16, BF16, F32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 1037), (3, 7), (5, 33), (64, 64), (130, 2050), (1000, 9)])
def test_no_dropout_changes_no_bit(m, n, dtype):
    """p = 0, p below its first step, and none at all: negative zeros, infinities and the smallest
    numbers come out as they went in, forward and back."""
    x = rand((m, n), 1, dtype)
    odd = torch.tensor([-0.0, math.inf, -math.inf, torch.finfo(dtype).smallest_normal, torch.finfo(dtype).max], device=x.device)
    small = torch.tensor([torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps], device=x.device)
    odd = torch.cat([odd, small, -3 * small]).to(dtype)
    x.view(-1)[:odd.numel()] = odd[:x.numel()]
    for drop in (None, L.Dropout(0.0, 1), L.Dropout(2.0 ** -18, 1)):
        assert same_bits(L.dropout(x, drop), x)
        assert same_bits(L.dropout_backward(x, drop)[0], x)
        assert same_bits(L.dropout(x, drop, residual=torch.zeros_like(x)), x + 0.0)


@HALVES
def test_every_half_passes_dropout(half):
    """All values of the type but NaN, kept with a factor of 1."""
    x = every_half(half).view(-1, 2).to("cuda:0")
    assert same_bits(L.dropout(x, None), x) and same_bits(L.dropout_backward(x, None)[0], x)


@HALVES
@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("m,n,k", [(6, 10, 7), (1, 9, 4), (9, 1, 3)])
def test_gradients_against_differences_of_each_element(m, n, k, act, half):
    """Every element of the layer's gradients, by differences of the 64-bit form at the same inputs
    and mask.  What an element may be off by is made of its own operands: the kernels' roundings
    (linear_reference.backward), the slope's change where pre was rounded, the differences' own error."""
    x, w, b, dy = rand((m, k), 1, half), rand((n, k), 2, half), rand((n,), 3, half), rand((m, n), 4, half)
    drop, ref = drops(0.25)
    scale, kept = R.keep(ref, m, n)
    pre = L.linear(x, w, b, pre=True)[1]
    got = L.linear_backward(dy, x, w, pre, act, drop, dbias=True)
    bounds = R.backward(dy, x, w, pre, act, ref)[2]
    xs = [t.double().cpu() for t in (x, w, b)]
    g = dy.double().cpu()
    v, h = xs[0] @ xs[1].t() + xs[2], 1e-4
    # (no element of v may cross RELU's corner, by its rounding or by a difference)
    moved = (pre.double().cpu() - v).abs()
    assert bool((v.abs() > moved + h * 8).all())

    def loss(x, w, b):
        return (R.dropped(R.act(act, x @ w.t() + b), ref) * g).sum().item()

    # second derivatives of the acts are at most 0.8, third ones 2, but for RELU's and none's, which are 0
    second, third = (0.0, 0.0) if act in ("none", "relu") else (0.81, 2.0)
    size = g.abs() * kept * scale
    slopes = size * second * moved
    absx, absw = xs[0].abs(), xs[1].abs()
    hides = {"dx": (slopes @ absw, size @ absw ** 3), "dw": (slopes.t() @ absx, size.t() @ absx ** 3),
             "dbias": (slopes.sum(0), size.sum(0))}
    terms = (size * R.act(act, v).abs()).sum().item()
    for which, (name, t) in enumerate(zip(("dx", "dw", "dbias"), got)):
        diff = torch.empty_like(xs[which])
        for at in range(diff.numel()):
            up, down = [t.clone() for t in xs], [t.clone() for t in xs]
            up[which].view(-1)[at] += h
            down[which].view(-1)[at] -= h
            diff.view(-1)[at] = (loss(*up) - loss(*down)) / (2 * h)
        rounded, cubes = hides[name]
        # a sum of up to 60 terms in 64 bits, twice, over 2 h
        bound = bounds[name][1] + rounded + h * h / 6 * third * cubes + (terms + 1) * 2.0 ** -53 * 64 / h
        R.close(t, diff, bound, name)
