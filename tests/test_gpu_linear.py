"""The linear layer's operators on the GPU against their 64-bit forms (tests/linear_reference.py)."""
import math

import pytest

torch = pytest.importorskip("torch")

import linear_reference as R  # noqa: E402
import mixed_precision_zero_amd as Z  # noqa: E402
from mixed_precision_zero_amd import linear as L  # noqa: E402
from linear_cases import PAIRS, PRODUCTS  # noqa: E402
from mixed_precision_zero_amd import matrix as M  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALVES = pytest.mark.parametrize("half", [F16, BF16], ids=["f16", "bf16"])
SEED, OFFSET = 0x9E3779B97F4A7C15, 0x1234567890


def rand(shape, seed, dtype=F16, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * sigma).to(dtype).to(DEV)


def ints(shape, seed, dtype=F16, top=3):
    """Small whole numbers: their products' sums are exact in FP32, whatever the order."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g).to(dtype).to(DEV)


def inside(t, before, extra, fill=math.nan):
    """t's values as columns of a wider buffer that holds `fill`: (buffer, view)."""
    rows, cols = t.shape
    flat = torch.full((rows * (cols + extra) + before + extra,), fill, dtype=t.dtype, device=t.device)
    view = flat[before:].as_strided((rows, cols), (cols + extra, 1))
    view.copy_(t)
    return flat, view


def untouched(flat, view, fill=math.nan):
    """Everything of flat but view still holds fill."""
    view.fill_(fill)
    same = torch.isnan(flat) if math.isnan(fill) else flat == fill
    assert bool(same.all())


def drops(p):
    return (L.Dropout(p, SEED, OFFSET), (p, SEED, OFFSET)) if p else (None, None)


def same_bits(a, b):
    kind = torch.int32 if a.dtype == F32 else torch.int16
    return a.dtype == b.dtype and a.shape == b.shape and bool((a.contiguous().view(kind) == b.contiguous().view(kind)).all())


# Sizes on both sides of every tile and split: single tokens, odd and ragged ones, few results over
# long sums, many results over short ones.
SIZES = [(1, 1, 1), (1, 8, 8), (1, 64, 64), (3, 5, 7), (1, 1000, 777), (2, 33, 65), (7, 130, 31), (16, 256, 512),
         (17, 100, 1000), (15, 4096, 64), (33, 63, 129), (64, 64, 64), (65, 127, 64), (100, 1000, 72), (128, 128, 4096),
         (129, 257, 136), (200, 72, 2056), (256, 512, 256), (257, 520, 200), (300, 300, 300), (513, 1030, 96),
         (1000, 24, 40), (40, 2000, 24), (640, 768, 64), (1, 2048, 8200), (5, 24, 16384), (50, 96, 8192)]


@HALVES
@pytest.mark.parametrize("m,n,k", SIZES)
def test_forward_sizes(m, n, k, half):
    """Whole numbers, so every sum is exact: the result is the exact one, rounded once."""
    x, w = ints((m, k), m + 7 * n + k, half), ints((n, k), m + n + 3 * k, half)
    want = x.double().cpu() @ w.double().cpu().t() + 0.0       # a sum that begins with 0 is never -0
    y, pre = L.linear(x, w)
    assert pre is None and same_bits(y.cpu(), want.to(half))
    y32, pre = L.linear(x, w, dtype=F32, pre=True)
    assert same_bits(y32.cpu(), want.float()) and same_bits(pre.cpu(), want.to(half))


@HALVES
@pytest.mark.parametrize("m,n,k", SIZES)
def test_backward_sizes(m, n, k, half):
    dy, x, w = ints((m, n), m, half), ints((m, k), n, half), ints((n, k), k, half)
    dx, dw, db = L.linear_backward(dy, x, w, dbias=True)
    d = dy.double().cpu()
    assert same_bits(dx.cpu(), (d @ w.double().cpu() + 0.0).to(half))
    assert same_bits(dw.cpu(), (d.t() @ x.double().cpu() + 0.0).to(half))
    assert same_bits(db.cpu(), (d.sum(0) + 0.0).to(half))


@HALVES
@pytest.mark.parametrize("kernel,shared,I,J,K", PRODUCTS)
def test_every_product_kernel(kernel, shared, I, J, K, half):
    """Each kernel, with and without shares of K, in the three products that take it: whole numbers,
    exact sums, the epilogue's bias and residual among them."""
    a, b = ints((J, K), 1, half, 2), ints((I, K), 2, half, 2)
    bias, res = ints((I,), 3, half, 9), ints((J, I), 4, half, 9)
    want = a.double() @ b.double().t() + 0.0
    y, pre = L.linear(a, b, bias, residual=res, act="relu", pre=True)
    v = want + bias.double()
    assert same_bits(pre, v.to(half)) and same_bits(y, (v.clamp(min=0) + res.double()).to(half))
    dx, _, _ = L.linear_backward(a, None, b.t().contiguous(), dw=False)
    assert same_bits(dx, want.to(half))
    dw = res.clone()
    L.linear_backward(a.t().contiguous(), b.t().contiguous(), None, dx=False, dw=dw, accumulate=True)
    assert same_bits(dw, (want + res.double()).to(half))


@HALVES
@pytest.mark.parametrize("m,n,k", [(1, 24576, 1000), (3, 50000, 400), (16, 24576, 6144), (16, 6144, 24576), (64, 6144, 8200),
                                   (33, 4099, 4105)])
def test_weights_read_once(m, n, k, half):
    """Few tokens by weights that are not kept in the caches, forward and back."""
    x, w, dy = ints((m, k), 1, half, 1), ints((n, k), 2, half, 1), ints((m, n), 3, half, 1)
    y, _ = L.linear(x, w)
    assert same_bits(y, (x.double() @ w.double().t() + 0.0).to(half))
    dx, _, _ = L.linear_backward(dy, None, w, dw=False)
    assert same_bits(dx, (dy.double() @ w.double() + 0.0).to(half))


@HALVES
@pytest.mark.parametrize("kernel,m,n,k", PAIRS)
def test_gradients_in_one_launch_and_in_two(kernel, m, n, k, half):
    """The three gradients together have the bits of each by itself, and the exact values."""
    dy, x, w = ints((m, n), 1, half, 2), ints((m, k), 2, half, 2), ints((n, k), 3, half, 2)
    db = ints((n,), 4, half, 9)
    d, want_b = dy.double(), db.double() + dy.double().sum(0)
    dx, dw, _ = L.linear_backward(dy, x, w)
    assert same_bits(dx, (d @ w.double() + 0.0).to(half))
    assert same_bits(dw, (d.t().contiguous() @ x.double() + 0.0).to(half))
    more, again = dw.clone(), db.clone()
    dx2, _, _ = L.linear_backward(dy, x, w, dw=more, dbias=again, accumulate=True)
    assert same_bits(dx2, dx) and same_bits(again, want_b.to(half))
    assert same_bits(more, (dw.double() + d.t().contiguous() @ x.double()).to(half))
    pre = rand((m, n), 5, half)
    drop = L.Dropout(0.2, 1)
    a = L.linear_backward(dy, x, w, pre, "gelu", drop, dbias=True)
    assert same_bits(a[0], L.linear_backward(dy, None, w, pre, "gelu", drop, dw=False)[0])
    assert same_bits(a[1], L.linear_backward(dy, x, None, pre, "gelu", drop, dx=False)[1])
    assert same_bits(a[2], L.linear_backward(dy, None, None, pre, "gelu", drop, dx=False, dw=False, dbias=True)[2])


@HALVES
@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("m,n,k", [(1, 50, 70), (37, 129, 260), (300, 264, 136)])
def test_forward_epilogue(m, n, k, act, half):
    x, w = rand((m, k), 1, half), rand((n, k), 2, half, 1.5 / math.sqrt(k))
    bias, res = rand((n,), 3, half, 0.5), rand((m, n), 4, half)
    for p, dtype in ((0.0, half), (0.25, half), (0.25, F32)):
        drop, ref = drops(p)
        r = res.to(dtype)
        y, pre = L.linear(x, w, bias, act, drop, r, dtype=dtype, pre=True)
        wy, wp, ey, ep = R.forward(x, w, bias, act, ref, r)
        R.close(y, wy, ey, f"y, p {p}")
        R.close(pre, wp, ep, "pre")


@HALVES
@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("m,n,k", [(1, 50, 70), (37, 129, 260), (300, 264, 136)])
def test_backward_epilogue(m, n, k, act, half):
    dy, x, w = rand((m, n), 1, half, 0.1), rand((m, k), 2, half), rand((n, k), 3, half, 0.1)
    pre = rand((m, n), 4, half, 2.0)
    for p in (0.0, 0.25):
        drop, ref = drops(p)
        got = dict(zip(("dx", "dw", "dbias"), L.linear_backward(dy, x, w, pre, act, drop, dbias=True)))
        want = R.backward(dy, x, w, pre, act, ref)[2]
        for name in want:
            R.close(got[name], *want[name], what=f"{name}, p {p}")


def every_half(half):
    """All finite values of the type, and the infinities."""
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(half)
    return v[~torch.isnan(v)]


@HALVES
@pytest.mark.parametrize("act", R.ACTS)
def test_acts_of_every_value(act, half):
    """act of each value of the type, through a product with 1, stored in FP32."""
    v = every_half(half)
    x, one = v.view(-1, 1).to(DEV), torch.ones(1, 1, dtype=half, device=DEV)
    y, _ = L.linear(x, one, act=act, dtype=F32)
    want = R.act(act, v.double())
    err = R.act_error(act, v.double()).view(-1, 1)
    R.close(y, want.view(-1, 1), err)
    nan, _ = L.linear(torch.full((3, 1), math.nan, dtype=half, device=DEV), one, act=act)
    assert bool(torch.isnan(nan).all())


@HALVES
@pytest.mark.parametrize("act", R.ACTS[1:])
def test_slopes_of_every_value(act, half):
    v = every_half(half).view(-1, 1).to(DEV)
    one = torch.ones(1, 1, dtype=half, device=DEV)
    dx, _, _ = L.linear_backward(torch.ones_like(v), w=one, pre=v, act=act, dw=False)
    d, bound, _ = R.backward(torch.ones_like(v), pre=v, act_name=act)
    R.close(dx, d, bound)
    dx, _, _ = L.linear_backward(torch.ones_like(v[:3]), w=one, pre=torch.full_like(v[:3], math.nan), act=act, dw=False)
    assert bool(torch.isnan(dx).all())


# ----------------------------------------------------------------------------------------
# dropout
# ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F16, BF16, F32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 8), (1, 1037), (3, 7), (2, 2048), (5, 33), (64, 64), (130, 2050), (1000, 9),
                                 (4097, 24)])
def test_dropout(m, n, dtype):
    x, bias, res = rand((m, n), 1, dtype), rand((n,), 2, dtype), rand((m, n), 3, dtype)
    for p, b, r in ((0.1, bias, res), (0.5, None, None), (0.0, bias, res), (0.999, None, res), (1.0, bias, res)):
        drop, ref = drops(p)
        y = L.dropout(x, drop, b, r)
        v = x.double().cpu() + (0 if b is None else b.double().cpu())
        want = R.dropped(v, ref)
        # the bias's addition and the scale are rounded to FP32
        err = want.abs() * 2 * R.U
        if r is not None:
            want = want + r.double().cpu()
            err = err + want.abs() * R.U
        R.close(y, want, err, f"p {p}")
        if p == 0.0 and dtype != F32 and b is None and r is None:
            assert same_bits(y, x)


@pytest.mark.parametrize("dtype", [F16, BF16, F32], ids=["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 1037), (3, 7), (2, 2048), (5, 33), (64, 64), (130, 2050), (3000, 9),
                                 (4097, 24), (700, 300)])
def test_dropout_backward(m, n, dtype):
    dy = rand((m, n), 5, dtype)
    old = rand((n,), 6, dtype)
    for p in (0.0, 0.3, 1.0):
        drop, ref = drops(p)
        dx, db = L.dropout_backward(dy, drop, dbias=True)
        want = R.dropped(dy.double().cpu(), ref)
        R.close(dx, want, want.abs() * R.U)
        err = (m + 1) * R.U * want.abs().sum(0)
        R.close(db, want.sum(0), err)
        more = old.clone()
        only, again = L.dropout_backward(dy, drop, dx=False, dbias=more, accumulate=True)
        assert only is None and again is more
        total = want.sum(0) + old.double().cpu()
        R.close(more, total, err + R.U * total.abs())
        inplace = dy.clone()
        assert L.dropout_backward(inplace, drop, dx=inplace)[0] is inplace and same_bits(inplace, dx)


@pytest.mark.parametrize("p", [2.0 ** -18, 2.0 ** -17, 3 * 2.0 ** -17, 1 - 2.0 ** -17, 1 - 2.0 ** -18, 0.25 + 2.0 ** -17])
def test_probabilities_between_steps(p):
    """The limit is rounded to the nearest of 65536 steps, ties to the even one."""
    x = torch.ones(200, 999, dtype=F32, device=DEV)
    y = L.dropout(x, L.Dropout(p, 5, 6))
    scale, k = R.keep((p, 5, 6), 200, 999)
    assert bool((y.cpu() == k.float() * scale).all())


def test_masks_of_seeds_offsets_and_counters():
    x = torch.ones(40, 100, dtype=F16, device=DEV)
    counter = torch.tensor([0], dtype=torch.int64, device=DEV)
    for seed, offset, c in ((0, 0, 0), ((1 << 64) - 1, (1 << 64) - 1, 0), (1, 1 << 32, 5), (1 << 32, 7, -1),
                            (3, (1 << 64) - 2, 3), (3, 0, -(1 << 63))):
        counter.fill_(c)
        o = (offset + c) % (1 << 64)
        want = R.keep((0.5, seed, o), 40, 100)[1]
        got = L.dropout(x, L.Dropout(0.5, seed, offset, counter))
        assert bool(((got != 0).cpu() == want).all())
        assert same_bits(got, L.dropout(x, L.Dropout(0.5, seed, o)))


@HALVES
def test_one_mask_everywhere(half):
    """The product's epilogue, its backward pass and dropout by itself drop the same elements,
    in every kernel, and a mask does not depend on the matrix's width or height."""
    full = R.keep((0.4, SEED, OFFSET), 600, 700)[1]
    drop = L.Dropout(0.4, SEED, OFFSET)
    for m, n in ((1, 700), (7, 33), (16, 64), (100, 300), (600, 700), (600, 8), (1, 1)):
        want = full[:m, :n]
        one = torch.ones(m, n, dtype=half, device=DEV)
        assert bool(((L.dropout(one, drop) != 0).cpu() == want).all())
        assert bool(((L.dropout_backward(one, drop)[0] != 0).cpu() == want).all())
        for k in (1, 64, 1000):
            y, _ = L.linear(torch.ones(m, k, dtype=half, device=DEV), torch.ones(n, k, dtype=half, device=DEV), dropout=drop)
            assert bool(((y != 0).cpu() == want).all())
        dx, _, _ = L.linear_backward(one, w=torch.eye(n, dtype=half, device=DEV), dropout=drop, dw=False)
        assert bool(((dx != 0).cpu() == want).all())
        y, _ = L.mxfp4_linear(torch.ones(m, 128, dtype=half, device=DEV),
                              M.mxfp4_quantize(torch.ones(n, 128, dtype=half, device=DEV)), dropout=drop)
        assert bool(((y != 0).cpu() == want).all())


@HALVES
def test_dropped_infinities_and_nan_are_zero(half):
    m, n = 50, 90
    k = R.keep((0.5, 1, 2), m, n)[1].to(DEV)
    drop = L.Dropout(0.5, 1, 2)
    for bad in (math.nan, math.inf, -math.inf):
        x = torch.where(k, 1.0, bad).to(half)
        assert bool((L.dropout(x, drop) == torch.where(k, 2.0, 0.0)).all())
        dx, db = L.dropout_backward(x, drop, dbias=True)
        assert bool((dx == torch.where(k, 2.0, 0.0)).all()) and bool((db == 2.0 * k.sum(0)).all())
        # the same values as a product's sums, and on their way back
        eye = torch.eye(n, dtype=half, device=DEV)
        res = torch.ones(m, n, dtype=half, device=DEV)
        y, _ = L.linear(torch.where(k, 1.0, 0.0).to(half), eye, dropout=drop, residual=res)
        assert bool((y == torch.where(k, 3.0, 1.0)).all())
        col = torch.tensor([[bad]], dtype=half, device=DEV)       # every sum is inf or NaN
        y, _ = L.linear(col.expand(m, 1).contiguous(), torch.ones(n, 1, dtype=half, device=DEV), dropout=drop)
        assert bool((y[~k] == 0).all()) and not bool(torch.isfinite(y[k]).any())
        dx, _, db = L.linear_backward(x, w=eye, dropout=drop, dw=False, dbias=True)
        assert bool((dx == torch.where(k, 2.0, 0.0)).all()) and bool((db == 2.0 * k.sum(0)).all())


@HALVES
def test_infinities_and_nan_reach_the_gradients(half):
    """As the step's overflow check needs: one in dy spreads over its row of dx, its rows of dw."""
    m, n, k = 70, 90, 40
    dy, x, w = rand((m, n), 1, half), rand((m, k), 2, half), rand((n, k), 3, half)
    for bad in (math.nan, math.inf):
        dy[33, 44] = bad
        dx, dw, db = L.linear_backward(dy, x, w, dbias=True)
        fine = torch.ones(m, dtype=torch.bool)
        fine[33] = False
        assert not bool(torch.isfinite(dx[33]).any()) and bool(torch.isfinite(dx[fine.to(DEV)]).all())
        assert not bool(torch.isfinite(dw[44]).any()) and not bool(torch.isfinite(db[44]))
        assert int((~torch.isfinite(dw)).sum()) == k and int((~torch.isfinite(db)).sum()) == 1


# ----------------------------------------------------------------------------------------
# layouts
# ----------------------------------------------------------------------------------------

@HALVES
@pytest.mark.parametrize("before,extra", [(0, 8), (8, 16), (1, 7), (3, 1), (2, 30), (4, 3)])
@pytest.mark.parametrize("m,n,k", [(5, 70, 130), (130, 100, 72), (300, 520, 264)])
def test_strides_and_alignment(m, n, k, before, extra, half):
    """Rows inside wider buffers, beginning anywhere: the bits of the contiguous call, and nothing
    around the results is touched (what surrounds the inputs is NaN)."""
    x, w, dy = rand((m, k), 1, half), rand((n, k), 2, half), rand((m, n), 3, half)
    pre, res, bias = rand((m, n), 4, half), rand((m, n), 5, half), rand((n,), 6, half)
    drop = L.Dropout(0.2, 3)
    y0, p0 = L.linear(x, w, bias, "gelu", drop, res, pre=True)
    g0 = L.linear_backward(dy, x, w, pre, "silu", drop, dbias=True)
    d0, e0 = L.dropout(dy, drop, bias, res), L.dropout_backward(dy, drop, dbias=True)
    put = lambda t: inside(t, before, extra)[1]
    new = lambda *s: inside(torch.empty(*s, dtype=half, device=DEV), before, extra)
    (fy, y), (fp, p), (fx, dx), (fw, dw), (fd, d) = new(m, n), new(m, n), new(m, k), new(n, k), new(m, n)
    b = inside(bias.view(1, n), before, extra)[1][0]
    L.linear(put(x), put(w), b, "gelu", drop, put(res), out=y, pre=p)
    assert same_bits(y, y0) and same_bits(p, p0)
    fb, db = new(1, n)
    L.linear_backward(put(dy), put(x), put(w), put(pre), "silu", drop, dx=dx, dw=dw, dbias=db[0])
    assert same_bits(dx, g0[0]) and same_bits(dw, g0[1]) and same_bits(db[0], g0[2])
    L.dropout(put(dy), drop, b, put(res), out=d)
    assert same_bits(d, d0)
    L.dropout_backward(put(dy), drop, dx=d, dbias=db[0])
    assert same_bits(d, e0[0]) and same_bits(db[0], e0[1])
    for f, v in ((fy, y), (fp, p), (fx, dx), (fw, dw), (fd, d), (fb, db)):
        untouched(f, v)


@HALVES
def test_slices_of_a_fused_buffer(half):
    """x and the result as columns of one array."""
    m, k, n = 90, 64, 48
    buf = rand((m, k + n + 32), 1, half)
    w = rand((n, k), 2, half)
    want, _ = L.linear(buf[:, :k].contiguous(), w)
    before = buf.clone()
    L.linear(buf[:, :k], w, out=buf[:, k:k + n])
    assert same_bits(buf[:, k:k + n], want)
    assert same_bits(buf[:, :k], before[:, :k]) and same_bits(buf[:, k + n:], before[:, k + n:])


@HALVES
@pytest.mark.parametrize("m", [4, 150])
def test_result_in_the_residual(m, half):
    x, w, res = rand((m, 200), 1, half), rand((130, 200), 2, half), rand((m, 130), 3, half)
    for dtype in (half, F32):
        r = res.to(dtype)
        want, _ = L.linear(x, w, residual=r, act="relu", dtype=dtype)
        got, _ = L.linear(x, w, residual=r, act="relu", out=r)
        assert got is r and same_bits(r, want)
    a = rand((m, 33), 4, half)
    want = L.dropout(a, L.Dropout(0.5, 1), residual=res[:, :33])
    r = res[:, :33].clone()
    assert same_bits(L.dropout(a, L.Dropout(0.5, 1), residual=r, out=r), want)
    want = L.dropout(a, L.Dropout(0.5, 1))
    assert same_bits(L.dropout(a, L.Dropout(0.5, 1), out=a), want)


@HALVES
@pytest.mark.parametrize("m,n,k", [(1, 30, 50), (70, 130, 72), (2000, 64, 64), (300, 520, 264)])
def test_accumulated_gradients(m, n, k, half):
    """Micro-batches added into the step's gradient: each call rounds once, from FP32."""
    dy, x = ints((m, n), 1, half), ints((m, k), 2, half)
    dw, db = ints((n, k), 3, half, 50), ints((n,), 4, half, 50)
    want = dw.double().cpu() + dy.double().cpu().t() @ x.double().cpu()
    wb = db.double().cpu() + dy.double().cpu().sum(0)
    L.linear_backward(dy, x, dx=False, dw=dw, dbias=db, accumulate=True)
    assert same_bits(dw.cpu(), want.to(half)) and same_bits(db.cpu(), wb.to(half))


@HALVES
def test_no_tokens(half):
    none, w = torch.empty(0, 40, dtype=half, device=DEV), rand((30, 40), 1, half)
    y, pre = L.linear(none, w, bias=rand((30,), 2, half), act="gelu", pre=True)
    assert y.shape == (0, 30) and pre.shape == (0, 30)
    dy = torch.empty(0, 30, dtype=half, device=DEV)
    dx, dw, db = L.linear_backward(dy, none, w, dbias=True)
    assert dx.shape == (0, 40) and not dw.any() and not db.any()
    dw, db = rand((30, 40), 3, half), rand((30,), 4, half)
    a, b = dw.clone(), db.clone()
    L.linear_backward(dy, none, dx=False, dw=dw, dbias=db, accumulate=True)
    assert same_bits(dw, a) and same_bits(db, b)
    assert L.dropout(dy, L.Dropout(0.5, 1)).shape == (0, 30)
    assert not L.dropout_backward(dy, None, dbias=True)[1].any()


@HALVES
def test_parts_of_the_gradients(half):
    """Any of the three by itself has the bits of the call for all."""
    m, n, k = 130, 70, 90
    dy, x, w, pre = rand((m, n), 1, half), rand((m, k), 2, half), rand((n, k), 3, half), rand((m, n), 4, half)
    for act in ("none", "gelu_tanh"):
        for drop in (None, L.Dropout(0.3, 9)):
            dx, dw, db = L.linear_backward(dy, x, w, pre, act, drop, dbias=True)
            assert same_bits(L.linear_backward(dy, None, w, pre, act, drop, dw=False)[0], dx)
            assert same_bits(L.linear_backward(dy, x, None, pre, act, drop, dx=False)[1], dw)
            got = L.linear_backward(dy, None, None, pre, act, drop, dx=False, dw=False, dbias=True)
            assert got[0] is None and got[1] is None and same_bits(got[2], db)


# ----------------------------------------------------------------------------------------
# the layer on 4-bit copies
# ----------------------------------------------------------------------------------------

@HALVES
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 48, 200), (1, 17000, 64), (9, 100, 333), (16, 520, 1024), (20, 100, 700),
                                   (33, 2000, 64), (64, 24, 512), (65, 130, 257), (300, 200, 128), (700, 3000, 256),
                                   (1500, 2500, 64)])
def test_mxfp4_linear(m, n, k, half):
    """The product's own sums (neox_mxfp4_product in FP32), taken through the epilogue."""
    x, w = M.mxfp4_quantize(rand((m, k), 1, half)), M.mxfp4_quantize(rand((n, k), 2, half, 1 / math.sqrt(k)))
    bias, res = rand((n,), 3, half), rand((m, n), 4, half)
    v = M.mxfp4_product(x, w, F32)
    assert same_bits(L.mxfp4_linear(x, w, dtype=F32, half=half)[0], v)
    assert same_bits(L.mxfp4_linear(x, w, half=half)[0], v.to(half))
    for act, p, dtype in (("gelu_tanh", 0.0, half), ("silu", 0.3, half), ("gelu", 0.3, F32), ("none", 0.1, F32), ("relu", 0.0, half)):
        drop, ref = drops(p)
        r = res.to(dtype)
        y, pre = L.mxfp4_linear(x, w, bias, act, drop, r, dtype=dtype, half=half, pre=True)
        s = v.double().cpu() + bias.double().cpu()
        es = s.abs() * R.U
        R.close(pre, s, es, "pre")
        scale, kept = R.keep(ref, m, n)
        want = torch.where(kept, R.act(act, s) * scale, torch.zeros((), dtype=s.dtype))
        err = (1.13 * es + R.act_error(act, s)) * scale + want.abs() * R.U
        want = want + r.double().cpu()
        R.close(y, want, err + want.abs() * R.U, act)


def test_mxfp4_linear_from_a_matrix():
    x, w = rand((30, 96), 1, BF16), M.mxfp4_quantize(rand((50, 96), 2, BF16))
    a, _ = L.mxfp4_linear(x, w, act="silu")
    b, _ = L.mxfp4_linear(M.mxfp4_quantize(x), w, act="silu")
    assert a.dtype == BF16 and same_bits(a, b)
    assert L.mxfp4_linear(x.half(), w)[0].dtype == F16 and L.mxfp4_linear(x.float(), w)[0].dtype == BF16


# ----------------------------------------------------------------------------------------
# how calls run
# ----------------------------------------------------------------------------------------

def test_conveniences_refuse_on_the_gpu():
    x, w = rand((4, 8), 1), rand((6, 8), 2)
    for f in (lambda: L.linear(x, w.bfloat16()), lambda: L.linear(x, rand((6, 9), 3)), lambda: L.linear(x.float(), w.float()),
              lambda: L.linear(x, w, act="tanh"), lambda: L.linear(x, w, bias=rand((5,), 1)),
              lambda: L.linear(x, w, residual=rand((4, 6), 1, F32)), lambda: L.linear(x, w, out=rand((4, 7), 1)),
              lambda: L.linear(x, w, dtype=F32, out=rand((4, 6), 1)), lambda: L.linear(x, w, pre=rand((4, 6), 1, F32)),
              lambda: L.linear(x.t(), w), lambda: L.linear_backward(rand((4, 6), 1), x, w, act="gelu"),
              lambda: L.linear_backward(rand((4, 6), 1), x), lambda: L.linear_backward(rand((4, 6), 1), None, w),
              lambda: L.linear_backward(rand((4, 6), 1), x, w, accumulate=True),
              lambda: L.linear_backward(rand((4, 6), 1), x, rand((6, 9), 1)),
              lambda: L.dropout(x, None, bias=rand((8,), 1, F32)), lambda: L.dropout(x, None, out=rand((4, 9), 1)),
              lambda: L.dropout_backward(x, None, dbias=True, accumulate=True),
              lambda: L.mxfp4_linear(x, M.mxfp4_quantize(rand((6, 9), 1))),
              lambda: L.Dropout(0.1, 0, 0, torch.zeros(2, dtype=torch.int64, device=DEV))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(Z.NeoxError):
        L.linear(x, w, out=torch.empty(4, 6, dtype=BF16, device=DEV))
    with pytest.raises(Z.NeoxError):
        L.linear(x, rand((8, 8), 1), out=x)


@HALVES
def test_runs_twice_alike(half):
    """No order of work changes a bit."""
    x, w, dy, pre = rand((700, 1000), 1, half), rand((500, 1000), 2, half), rand((700, 500), 3, half), rand((700, 500), 4, half)
    drop = L.Dropout(0.1, 1)
    first = [L.linear(x, w, act="gelu", dropout=drop)[0], *L.linear_backward(dy, x, w, pre, "gelu", drop, dbias=True)]
    for _ in range(3):
        again = [L.linear(x, w, act="gelu", dropout=drop)[0], *L.linear_backward(dy, x, w, pre, "gelu", drop, dbias=True)]
        assert all(same_bits(a, b) for a, b in zip(first, again))


def test_another_stream():
    x, w = rand((300, 4096), 1), rand((64, 4096), 2)
    want = L.linear(x, w, act="silu")[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a = x + 0
        got = L.linear(a, w, act="silu")[0]
    s.synchronize()
    assert same_bits(got, want)


@HALVES
def test_two_streams_at_once(half):
    """Calls that overlap take workspaces of their own."""
    cases = []
    for i, (m, n, k) in enumerate([(387, 1001, 999), (128, 128, 16384)]):
        dy, x, w, pre = rand((m, n), 10 + i, half), rand((m, k), 20 + i, half), rand((n, k), 30 + i, half), rand((m, n), 40 + i, half)
        drop = L.Dropout(0.1, i)

        def run(dy=dy, x=x, w=w, pre=pre, drop=drop):
            return [L.linear(x, w, act="gelu", dropout=drop, residual=dy)[0],
                    *L.linear_backward(dy, x, w, pre, "gelu", drop, dbias=True)]
        cases.append((run, run(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (run, _, stream) in enumerate(cases):
            with torch.cuda.stream(stream):
                got[i].append(run())
    torch.cuda.synchronize()
    for i, (_, want, _) in enumerate(cases):
        assert all(same_bits(a, b) for g in got[i] for a, b in zip(g, want))


def test_offsets_beyond_32_bits():
    """Results, gradients and masks of more than 2^32 elements: their last rows as well as their
    first; and sums over a million tokens."""
    m, n, k = (1 << 20) + 3, 4100, 24
    x, w = ints((m, k), 1, BF16, 1), ints((n, k), 2, BF16, 1)
    res = torch.ones(m, n, dtype=BF16, device=DEV)
    drop = L.Dropout(0.5, 5, 6)
    y, pre = L.linear(x, w, dropout=drop, residual=res, out=res, pre=True)
    for first in (0, (1 << 31) // n - 1, (1 << 32) // n - 1, m - 2):
        v = x[first:first + 2].double().cpu() @ w.double().cpu().t() + 0.0
        keep = R.draws(5, 6, 2, n, first) >= 32768
        assert same_bits(pre[first:first + 2].cpu(), v.to(BF16))
        assert same_bits(y[first:first + 2].cpu(), (torch.where(keep, v * 2, 0.0) + 1).to(BF16))
    dy = pre                                            # whole numbers of up to 24, few of them large
    dx, dw, db = L.linear_backward(dy, x, w, dbias=True)
    want = torch.zeros(n, k, dtype=torch.float64, device=DEV)
    bias = torch.zeros(n, dtype=torch.float64, device=DEV)
    for a in range(0, m, 1 << 16):
        d = dy[a:a + (1 << 16)].double()
        want += d.t().contiguous() @ x[a:a + (1 << 16)].double()
        bias += d.sum(0)
        if a == 0 or a + (1 << 16) >= m:
            assert same_bits(dx[a:a + (1 << 16)], (d @ w.double() + 0.0).to(BF16))
    assert float(want.abs().max()) < 2 ** 24            # so FP32's sums are exact
    assert same_bits(dw, want.to(BF16)) and same_bits(db, bias.to(BF16))
    del dy, pre, y, res
    x = torch.ones(70001, 70001, dtype=F16, device=DEV)
    y = L.dropout(x, drop, out=x)
    for first in (0, 30677, 30678, 61356, 70000):
        keep = R.draws(5, 6, 1, 70001, first) >= 32768
        assert bool(((y[first:first + 1] != 0).cpu() == keep).all())
    dx, db = L.dropout_backward(y, L.Dropout(0.0, 0), dx=False, dbias=True)
    kept = (y != 0).sum(0)
    assert same_bits(db, (2.0 * kept).to(F16))


@pytest.mark.parametrize("m,n,k", [(1 << 24, 8, 8), (1, 1 << 22, 16), (3, 16, 1 << 22)])
def test_longest_sides(m, n, k):
    """Each side at its limit: first, last and middle rows."""
    x, w, dy = ints((m, k), 1, BF16, 1), ints((n, k), 2, BF16, 1), ints((m, n), 3, BF16, 1)
    y, _ = L.linear(x, w, dtype=F32)
    dx, _, db = L.linear_backward(dy, None, w, dw=False, dbias=True)
    for rows in (slice(0, 2), slice(m // 2, m // 2 + 2), slice(max(0, m - 2), m)):
        assert same_bits(y[rows], (x[rows].double() @ w.double().t() + 0.0).float())
        assert same_bits(dx[rows], (dy[rows].double() @ w.double() + 0.0).to(BF16))
    assert same_bits(db, (dy.sum(0, dtype=torch.float64) + 0.0).to(BF16))
    if m > 1:
        _, dw, _ = L.linear_backward(dy, x, None, dx=False)
        want = torch.zeros(n, k, dtype=torch.float64, device=DEV)
        for a in range(0, m, 1 << 20):
            want += dy[a:a + (1 << 20)].double().t().contiguous() @ x[a:a + (1 << 20)].double()
        assert same_bits(dw, (want + 0.0).to(BF16))


def test_rows_of_any_length():
    """Dropout of rows that are taken as stripes and of rows that are taken in a row of all threads."""
    for n in list(range(1, 40)) + [63, 64, 65, 127, 130, 255, 256, 257, 1000, 1040, 2047, 2050, 4096, 6150]:
        m = max(3, 20000 // n)
        x, b, r = rand((m, n), n, F16), rand((n,), 2, F16), rand((m, n), 3, F16)
        want = R.dropped(x.double().cpu() + b.double().cpu(), (0.3, n, 7))
        y = L.dropout(x, L.Dropout(0.3, n, 7), b, r)
        err = want.abs() * 2 * R.U
        want = want + r.double().cpu()
        R.close(y, want, err + want.abs() * R.U, f"{m} x {n}")


def test_long_sums():
    """A million elements of K: exact, whole numbers of -1 to 1."""
    k = (1 << 20) + 8
    x, w = ints((5, k), 1, BF16, 1), ints((70, k), 2, BF16, 1)
    y, _ = L.linear(x, w, dtype=F32)
    assert same_bits(y, (x.double() @ w.double().t() + 0.0).float())


def test_captured_and_replayed():
    """A layer and its gradients in one graph: replays draw new masks from a counter that the graph
    itself moves on, and give the eager calls' bits, whatever else ran between."""
    m, n, k = 130, 264, 1000
    x, w, dy, bias, res = rand((m, k), 1), rand((n, k), 2, F16, 0.05), rand((m, n), 3), rand((n,), 4), rand((m, n), 5)
    counter = torch.zeros(1, dtype=torch.int64, device=DEV)
    drop = L.Dropout(0.2, 77, 5, counter)

    def step():
        y, pre = L.linear(x, w, bias, "gelu", drop, res, pre=True)
        grads = L.linear_backward(dy, x, w, pre, "gelu", drop, dbias=True)
        d = L.dropout(y, drop, residual=res)
        return [y, pre, *grads, d, *L.dropout_backward(d, drop, dbias=True)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
        counter += 1
    for i in range(4):
        counter.fill_(i * 3)
        x.copy_(rand((m, k), 100 + i))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert int(counter) == i * 3 + 1
        counter.fill_(i * 3)
        eager = step()
        assert all(same_bits(a, b) for a, b in zip(outs, eager)), i
        plain = L.linear(x, w, bias, "gelu", L.Dropout(0.2, 77, 5 + i * 3), res)[0]
        assert same_bits(plain, outs[0])


def test_gradients_against_differences():
    """The whole layer's gradients, by differences of the 64-bit form at the same inputs and mask."""
    m, n, k = 6, 10, 7
    x, w, b = rand((m, k), 1, F32).half(), rand((n, k), 2, F32).half(), rand((n,), 3, F32).half()
    dy = rand((m, n), 4, F32).half()
    drop, ref = drops(0.25)
    for act in R.ACTS[1:]:
        pre = L.linear(x, w, b, pre=True)[1]
        dx, dw, db = L.linear_backward(dy, x, w, pre, act, drop, dbias=True)

        def loss(x, w, b):
            v = x @ w.t() + b
            return float((R.dropped(R.act(act, v), ref) * dy.double().cpu()).sum())

        xs = [t.double().cpu() for t in (x, w, b)]
        for got, which in ((dx, 0), (dw, 1), (db, 2)):
            h = 1e-6
            for at in range(0, xs[which].numel(), 5):
                up, down = [t.clone() for t in xs], [t.clone() for t in xs]
                up[which].view(-1)[at] += h
                down[which].view(-1)[at] -= h
                diff = (loss(*up) - loss(*down)) / (2 * h)
                # pre and d are rounded to half on the way (2^-11 each, slopes change by at most 1 for
                # each unit of pre), over sums of at most 10 terms of up to 3 x 3 x 1.34
                assert abs(float(got.reshape(-1)[at]) - diff) < 2.0 ** -11 * 10 * 3 * 3 * 1.34 * 6, (act, which, at)


def test_layers_around_the_step():
    """Two layers of a model trained as the library is meant to be used: forward on the half
    weights the step writes, gradients accumulated over two micro-batches straight into the step's
    flat gradient, one AdamW step; the new half weights, as a 4-bit copy, serve a token."""
    h, f, tokens = 64, 160, 96
    shapes = [(f, h), (f,), (h, f), (h,)]
    numel = [math.prod(s) for s in shapes]
    total = sum(numel)
    master = torch.randn(total, generator=torch.Generator().manual_seed(1)).to(DEV) * 0.05
    half, grad = master.half(), torch.zeros(total, dtype=F16, device=DEV)
    m, v = torch.zeros_like(master), torch.zeros_like(master)
    scale = 64.0
    cfg = Z.neox_zero1_default_config(clip_norm=1.0, init_scale=scale, scaler_mode=Z.NEOX_SCALER_STATIC)
    segs, parts, grads, off = [], [], [], 0
    for s, c in zip(shapes, numel):
        cut = slice(off, off + c)
        segs.append(Z.segment(grad[cut], half[cut], master[cut], m[cut], v[cut], len(s) > 1))
        parts.append(half[cut].view(s))
        grads.append(grad[cut].view(s))
        off += c
    opt = Z.Zero1(cfg, segs)
    w1, b1, w2, b2 = parts
    g1, gb1, g2, gb2 = grads

    want = [torch.zeros(s, dtype=torch.float64) for s in shapes]
    bound = [torch.zeros(s, dtype=torch.float64) for s in shapes]
    for micro in range(2):
        x, target = rand((tokens, h), 10 + micro), rand((tokens, h), 20 + micro)
        drop = L.Dropout(0.1, 3, micro)
        a, pre = L.linear(x, w1, b1, "gelu_tanh", pre=True)
        y, _ = L.linear(a, w2, b2, dropout=drop, residual=x)
        dy = ((y.float() - target.float()) * (scale / tokens)).half()
        da, _, _ = L.linear_backward(dy, a, w2, dropout=drop, dw=g2, dbias=gb2, accumulate=True)
        dx, _, _ = L.linear_backward(da, x, w1, pre, "gelu_tanh", dw=g1, dbias=gb1, accumulate=True)
        assert dx.shape == x.shape
        for i, (args, kw) in ((2, ((dy, a, w2), dict(drop=(0.1, 3, micro)))),
                              (0, ((da, x, w1), dict(pre=pre, act_name="gelu_tanh")))):
            out = R.backward(*args, **kw)[2]
            for j, name in ((i, "dw"), (i + 1, "dbias")):
                g, e = out[name]
                want[j] += g
                # what was there before is rounded again by this call
                bound[j] += e + R.half_step(F16) * (want[j].abs() + bound[j]) if micro == 0 else e
    for g, wt, e in zip(grads, want, bound):
        R.close(g, wt, e)
    old = master.clone()
    opt.step(lr=1e-3)
    torch.cuda.synchronize()
    st = opt.state()
    assert st.step == 1 and abs(st.last_grad_norm - float((grad.double() / scale).norm())) < 1e-4 * st.last_grad_norm
    assert bool((master != old).any()) and same_bits(half, master.half())

    token = rand((1, h), 30)
    c1, c2 = M.mxfp4_quantize(w1), M.mxfp4_quantize(w2)
    a, _ = L.mxfp4_linear(token, c1, b1, "gelu_tanh")
    y, _ = L.mxfp4_linear(a, c2, b2, residual=token)
    wa = R.act("gelu_tanh", M.mxfp4_product(M.mxfp4_quantize(token), c1, F32).double().cpu() + b1.double().cpu())
    R.close(a, wa, wa.abs() * 1e-5 + 1e-6)
    wy = M.mxfp4_product(M.mxfp4_quantize(a), c2, F32).double().cpu() + b2.double().cpu() + token.double().cpu()
    R.close(y, wy, wy.abs() * 1e-6 + 1e-6)
    opt.close()
