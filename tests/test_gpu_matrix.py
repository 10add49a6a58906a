"""The matrix operators on the GPU against their 64-bit forms (tests/matrix_reference.py)."""
import math

import pytest

torch = pytest.importorskip("torch")

import matrix_reference as R  # noqa: E402
import mixed_precision_zero_amd as Z  # noqa: E402
from mixed_precision_zero_amd import matrix as M  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=["f32", "f16", "bf16"])


def rand(shape, seed, dtype=F32, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * sigma).to(dtype).to(DEV)


def padded(t, extra, fill):
    """t's values in a wider buffer: (buffer, view).  The rest of the buffer holds `fill`."""
    buf = torch.full((*t.shape[:-1], t.shape[-1] + extra), fill, dtype=t.dtype, device=t.device)
    buf[..., :t.shape[-1]] = t
    return buf, buf[..., :t.shape[-1]]


# ----------------------------------------------------------------------------------------
# orthogonalisation
# ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 9), (9, 1), (3, 5), (31, 33), (64, 64), (65, 63), (128, 128),
                                       (129, 127), (40, 700), (700, 40), (130, 513), (513, 257), (300, 1000), (520, 1100),
                                       (1300, 600), (60, 2100), (5000, 70), (200, 2500)])
def test_orthogonalize_sizes(rows, cols):
    x = rand((rows, cols), rows * 1000 + cols)
    R.check_orth(M.orthogonalize(x), x)


@TYPES
@pytest.mark.parametrize("out", [F32, F16, BF16], ids=["f32", "f16", "bf16"])
def test_orthogonalize_types_and_scale(dtype, out):
    x = rand((75, 203), 5, dtype, 1e-3)
    R.check_orth(M.orthogonalize(x, dtype=out, scale=0.25), x, scale=0.25)


@pytest.mark.parametrize("kind", ["rank1", "low", "decay", "flat", "tiny", "huge"])
def test_orthogonalize_spectra(kind):
    n = 192
    u, v = torch.linalg.qr(rand((n, n), 1).cpu())[0], torch.linalg.qr(rand((n, n), 2).cpu())[0]
    s = {"rank1": torch.tensor([1.0] + [0.0] * (n - 1)), "low": torch.tensor([1.0] * 8 + [0.0] * (n - 8)),
         "decay": torch.logspace(0, -4, n), "flat": torch.ones(n), "tiny": torch.ones(n) * 1e-4,
         "huge": torch.ones(n) * 1e30}[kind]
    x = (u @ torch.diag(s) @ v).to(DEV)
    R.check_orth(M.orthogonalize(x), x)


@pytest.mark.parametrize("shape", [(90, 140), (530, 1065)], ids=["single", "pairs"])
@pytest.mark.parametrize("coef", [[(1.5, -0.5, 0.0)] * 8, [(3.4445, -4.7750, 2.0315)], [(15 / 8, -10 / 8, 3 / 8)] * 3,
                                  [(4.0, -6.0, 3.0), (2.0, -1.5, 0.5)]])
def test_orthogonalize_steps(coef, shape):
    x = rand(shape, 3)
    R.check_orth(M.orthogonalize(x, cfg=M.neox_ns_default_config(coef=coef)), x, coef=coef)


@pytest.mark.parametrize("shape", [(5, 70, 33), (2, 3, 48, 200), (40, 64, 64), (0 + 1, 1, 7, 300)])
def test_orthogonalize_batches_are_independent(shape):
    """Each matrix of a batch has the bits it has alone."""
    x = rand(shape, 11)
    got = M.orthogonalize(x)
    flat, one = got.reshape(-1, *shape[-2:]), x.reshape(-1, *shape[-2:])
    for i in range(one.shape[0]):
        assert torch.equal(flat[i], M.orthogonalize(one[i].contiguous()))
    R.check_orth(flat[-1], one[-1])


def test_orthogonalize_strides_and_surroundings():
    """Row and matrix strides on both sides, an odd start, and nothing else written."""
    x = rand((3, 37, 61), 21, BF16)
    buf, view = padded(x, 7, math.nan)
    out, oview = padded(torch.zeros(3, 37, 61, dtype=F16, device=DEV), 9, 5.0)
    got = M.orthogonalize(view, out=oview)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(oview, M.orthogonalize(x, dtype=F16))
    assert (out[..., 61:] == 5.0).all() and torch.isnan(buf[..., 61:]).all()
    # every second matrix, starting one element into a buffer
    flat = torch.full((1 + 4 * 37 * 61,), 9.0, dtype=F32, device=DEV)
    tgt = flat[1:].view(4, 37, 61)[::2]
    M.orthogonalize(x[:2].contiguous(), out=tgt)
    assert torch.equal(tgt.contiguous(), M.orthogonalize(x[:2].contiguous(), dtype=F32))
    rest = flat[1:].view(4, 37, 61)[1::2]
    assert (rest == 9.0).all() and flat[0] == 9.0


@pytest.mark.parametrize("rows,heads,width", [(48, 6, 16), (300, 3, 130), (700, 2, 75)])
def test_orthogonalize_side_by_side_in_place(rows, heads, width):
    """A projection's heads: column blocks of one matrix, whose rows lie between each other's."""
    w = rand((rows, heads * width + 5), rows, BF16)
    keep = w.clone()
    blocks = w[:, :heads * width].view(rows, heads, width).transpose(0, 1)
    want = M.orthogonalize(blocks.contiguous())
    M.orthogonalize(blocks, out=blocks)
    assert torch.equal(blocks, want)
    assert torch.equal(w[:, heads * width:], keep[:, heads * width:])


def test_orthogonalize_in_place():
    x = rand((4, 150, 90), 31)
    want = M.orthogonalize(x)
    M.orthogonalize(x, out=x)
    assert torch.equal(x, want)


def test_orthogonalize_zero_and_non_finite():
    x = rand((5, 70, 130), 41)
    keep = M.orthogonalize(x)
    x[1] = 0
    x[2, 3, 4] = math.nan
    x[3, 69, 129] = math.inf
    got = M.orthogonalize(x)
    assert (got[1] == 0).all() and torch.isnan(got[2]).all() and torch.isnan(got[3]).all()
    assert torch.equal(got[0], keep[0]) and torch.equal(got[4], keep[4])
    one = torch.tensor([[math.nan]], device=DEV)
    assert torch.isnan(M.orthogonalize(one)).all()


@pytest.mark.parametrize("rows,cols", [(1500, 2900), (4200, 4400), (5000, 1030), (2304, 2304)])
def test_orthogonalize_large(rows, cols):
    """Many tiles of every kind (whole ones, quarters, cut by the edge), against 64 bits on the
    GPU."""
    x = rand((rows, cols), 51, BF16)
    got = M.orthogonalize(x, dtype=F32).double()
    g = x.double()
    if rows > cols:
        g, got = g.t().contiguous(), got.t()
    g = g / (torch.linalg.vector_norm(g) + 1e-7)
    for a, b, c in R.COEF:
        p = g @ g.t().contiguous()
        g = a * g + (b * p + c * (p @ p)) @ g
    # FP16 roundings: below 2^-9 of the norm for every spectrum simulated
    assert float((got - g).norm() / g.norm()) < 2.0 ** -9


def test_orthogonalize_refusals():
    x = rand((4, 6), 1)
    with pytest.raises(ValueError):
        M.orthogonalize(x.cpu())
    with pytest.raises(ValueError):
        M.orthogonalize(x.t())
    with pytest.raises(ValueError):
        M.orthogonalize(x.double())
    with pytest.raises(ValueError):
        M.orthogonalize(x, out=torch.empty(6, 4, device=DEV))
    with pytest.raises(ValueError):
        M.orthogonalize(x[0])
    with pytest.raises(ValueError):
        M.orthogonalize(rand((2, 3, 4, 6), 2)[:, :2])
    with pytest.raises(Z.NeoxError):
        M.orthogonalize(x[:0])
    with pytest.raises(Z.NeoxError):
        M.orthogonalize(x, out=x.view(-1)[:24].view(4, 6), cfg=M.neox_ns_default_config(steps=99))


# ----------------------------------------------------------------------------------------
# MXFP4
# ----------------------------------------------------------------------------------------

def planted(rows, cols, dtype, seed):
    """Values over many binades with ties, signed zeros, zero blocks, subnormals, the largest
    values, infinities and NaN planted."""
    x = rand((rows, cols), seed).cpu()
    x = x * torch.exp2(torch.randint(-20, 12, (rows, 1), generator=torch.Generator().manual_seed(seed)).float())
    flat = x.view(-1)
    n = flat.numel()
    fi = torch.finfo(dtype)
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.0, 7.9, -0.25, -0.75, -5.0, -7.0, 0.0, -0.0, 4.0]
    for i, v in enumerate(ties * 3):
        if n > 64 + i:
            flat[64 + i] = v
    if rows > 2 and cols >= 64:
        x[1, 32:64] = 0.0
        x[1, 33] = -0.0
        x[2, :32] = fi.smallest_normal * 2.0 ** -3 * torch.arange(32)
    if rows > 6:
        x[4, cols // 2] = math.inf
        x[5, 0] = math.nan
        x[6, -1] = -math.inf
    if rows > 8:
        x[7, 0] = fi.max
        x[8, -1] = -fi.max
    return x.to(dtype).to(DEV)


SHAPES = [(1, 1), (1, 31), (3, 32), (5, 33), (9, 64), (10, 129), (17, 256), (64, 1000), (33, 4097), (130, 300)]


@TYPES
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("extra", [0, 3], ids=["dense", "ld"])
@pytest.mark.parametrize("transpose", [False, True], ids=["rows", "transpose"])
def test_quantize_bits(dtype, rows, cols, extra, transpose):
    x = planted(rows, cols, dtype, rows * 7 + cols)
    src = padded(x, extra, 77.0)[1] if extra else x
    q = M.mxfp4_quantize(src, transpose=transpose)
    codes, scales = R.mx_quantize(x.t() if transpose else x)
    assert torch.equal(q.scales.cpu(), scales)
    assert torch.equal(q.codes.cpu(), codes)


@TYPES
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dequantize_bits(dtype, rows, cols):
    """Any codes and scales, not only the quantiser's; nothing beside the matrix is written."""
    g = torch.Generator().manual_seed(rows + cols)
    k = -(-cols // 128) * 128
    q = M.MXFP4(torch.randint(0, 256, (rows, k // 2), generator=g, dtype=torch.uint8).to(DEV),
                torch.randint(0, 256, (rows, k // 32), generator=g, dtype=torch.uint8).to(DEV), rows, cols)
    # FP32 cannot hold 6 * 2^127: it reads as inf, as rounding to FP32 says
    want = R.mx_values(q.codes, q.scales, cols).to(F32).to(dtype)
    buf, view = padded(torch.zeros(rows, cols, dtype=dtype, device=DEV), 5, 3.0)
    M.mxfp4_dequantize(q, out=view)
    got = M.mxfp4_dequantize(q, dtype)
    for t in (got.cpu(), view.cpu()):
        assert torch.equal(torch.isnan(t), torch.isnan(want))
        ok = ~torch.isnan(want)
        assert torch.equal(t[ok], want[ok]) and torch.equal(torch.signbit(t[ok]), torch.signbit(want[ok]))
    assert (buf[:, cols:] == 3.0).all()


def test_copies_beyond_32_bit_offsets():
    """A matrix of more than 2^32 elements, by its first and last rows."""
    rows, cols = 33_000, 131_200
    x = torch.empty(rows, cols, dtype=F16, device=DEV)
    x.view(-1)[:1 << 20] = rand((1 << 20,), 1, F16)
    x[-40:] = rand((40, cols), 2, F16)
    q = M.mxfp4_quantize(x)
    back = M.mxfp4_dequantize(q, F16)
    codes, scales = R.mx_quantize(x[-40:])
    assert torch.equal(q.codes[-40:].cpu(), codes) and torch.equal(q.scales[-40:].cpu(), scales)
    assert torch.equal(back[-40:].cpu(), R.mx_values(codes, scales, cols).to(F16))
    del back
    t = M.mxfp4_quantize(x, transpose=True)
    assert torch.equal(t.scales[:, rows // 32].cpu(), R.mx_quantize(x[rows // 32 * 32:].t())[1][:, 0])
    y = M.mxfp4_product(M.MXFP4(q.codes[-40:], q.scales[-40:], 40, cols), M.MXFP4(q.codes[-9:], q.scales[-9:], 9, cols), F32)
    a = R.mx_values(q.codes[-40:], q.scales[-40:], cols)
    assert ((y.double().cpu() - a @ a[-9:].t()).abs() <= product_bound(a, a[-9:], cols)).all()


def test_more_rows_than_one_launch_takes():
    """A transposed copy and a product of few rows with 2^22 and some rows: the rows of each
    launch, its first and last ones, against the same rows alone."""
    n = (1 << 22) + 19
    x = rand((3, 4099), 6, BF16).repeat(1, n // 4099 + 1)[:, :n].contiguous()
    t = M.mxfp4_quantize(x, transpose=True)
    for r0, r1 in ((0, 300), ((1 << 22) - 150, (1 << 22) + 19)):
        codes, scales = R.mx_quantize(x[:, r0:r1].t())
        assert torch.equal(t.codes[r0:r1].cpu(), codes) and torch.equal(t.scales[r0:r1].cpu(), scales)
    a = M.mxfp4_quantize(rand((2, 3), 8, BF16))
    y = M.mxfp4_product(a, t, dtype=F32)
    for r0, r1 in ((0, 300), ((1 << 22) - 150, (1 << 22) + 19)):
        part = M.MXFP4(t.codes[r0:r1].contiguous(), t.scales[r0:r1].contiguous(), r1 - r0, 3)
        assert torch.equal(y[:, r0:r1], M.mxfp4_product(a, part, dtype=F32))
        want = R.mx_values(a.codes, a.scales, 3) @ R.mx_values(part.codes, part.scales, 3).t()
        # three products of numbers with two significant bits each: exact unless scales differ by
        # more than 2^20, else three FP32 roundings of at most the sum of magnitudes
        top = R.mx_values(a.codes, a.scales, 3).abs() @ R.mx_values(part.codes, part.scales, 3).abs().t()
        assert ((y[:, r0:r1].double().cpu() - want).abs() <= 3 * 2.0 ** -24 * top).all()


def test_quantize_leaves_what_is_behind():
    x = rand((13, 100), 3)
    nc, ns = M.neox_mxfp4_layout(13, 100)
    codes = torch.full((nc + 64,), 0xAB, dtype=torch.uint8, device=DEV)
    scales = torch.full((ns + 64,), 0xCD, dtype=torch.uint8, device=DEV)
    M.neox_mxfp4_quantize(x.data_ptr(), M.NEOX_F32, 13, 100, 100, 0, codes.data_ptr(), scales.data_ptr(),
                          Z.current_stream_ptr())
    assert (codes[nc:] == 0xAB).all() and (scales[ns:] == 0xCD).all()


PRODUCTS = [(1, 1, 1), (1, 17, 129), (2, 16, 128), (3, 300, 257), (16, 128, 640), (17, 129, 384), (33, 257, 640),
            (64, 64, 32), (127, 200, 1000), (130, 131, 513), (300, 520, 2080)]


def product_bound(a, b, k):
    """k products, each exact in FP32 (two 4-bit values and a power of two), added in FP32 in
    some order: at most k additions, each off by half a step of a partial sum, which the sum of
    magnitudes bounds; twice that, as the matrix units may drop bits below the largest term of a
    group instead of rounding them."""
    return 2 * k * 2.0 ** -24 * (a.abs() @ b.abs().t())


@TYPES
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(dtype, m, n, k):
    x, w = rand((m, k), m + k), rand((n, k), n + k, sigma=0.02)
    qx, qw = M.mxfp4_quantize(x), M.mxfp4_quantize(w)
    a, b = R.mx_values(qx.codes, qx.scales, k), R.mx_values(qw.codes, qw.scales, k)
    want = a @ b.t()
    buf, view = padded(torch.zeros(m, n, dtype=dtype, device=DEV), 3, 7.0)
    M.mxfp4_product(qx, qw, out=view)
    got = M.mxfp4_product(qx, qw, dtype)
    assert torch.equal(got, view) and (buf[:, n:] == 7.0).all()
    err = (got.double().cpu() - want).abs()
    f = product_bound(a, b, k)
    u = torch.finfo(dtype).eps / 2
    tol = f + u * (want.abs() + f) + torch.finfo(dtype).smallest_normal * u
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("m,n,k", [(5, 40, 96), (12, 40000, 300), (60, 9000, 700), (16, 5000, 1500), (31, 16500, 600), (64, 200, 256), (150, 260, 4000),
                                   (4200, 4300, 200), (2500, 9000, 130), (700, 700, 64)])
def test_product_is_exact_on_small_integers(m, n, k):
    """Values of {0, +-1, +-2, +-4} at scales that make every sum an integer below 2^24 have
    one right answer."""
    g = torch.Generator().manual_seed(m)
    vals = torch.tensor([0.0, 1.0, 2.0, 4.0, -1.0, -2.0, -4.0])
    x = vals[torch.randint(0, 7, (m, k), generator=g)]
    w = vals[torch.randint(0, 7, (n, k), generator=g)]
    x[:, ::32] = 4.0
    w[:, ::32] = -4.0
    got = M.mxfp4_product(M.mxfp4_quantize(x.to(DEV)), M.mxfp4_quantize(w.to(DEV)), F32)
    assert torch.equal(got.cpu().double(), x.double() @ w.double().t())


@pytest.mark.parametrize("m,n,k", [(3, 50, 200), (140, 200, 700)])
def test_product_scales_and_nan(m, n, k):
    """Every block of its own scale, over 40 binades; a NaN block reaches its row (or column) of
    the result and nothing else."""
    g = torch.Generator().manual_seed(9)
    kb = -(-k // 128) * 4
    qs = []
    for rows in (m, n):
        q = M.mxfp4_quantize(rand((rows, k), rows))
        live = -(-k // 32)
        s = torch.randint(107, 148, (rows, kb), generator=g, dtype=torch.uint8)
        q.scales[:, :live] = s[:, :live].to(DEV)
        qs.append(q)
    a, b = (R.mx_values(q.codes, q.scales, k) for q in qs)
    got = M.mxfp4_product(*qs, F32).double().cpu()
    assert ((got - a @ b.t()).abs() <= product_bound(a, b, k)).all()
    qs[0].scales[1, 2] = 255
    qs[1].scales[n - 1, 0] = 255
    bad = M.mxfp4_product(*qs, F32).double().cpu()
    hit = torch.zeros(m, n, dtype=torch.bool)
    hit[1] = True
    hit[:, n - 1] = True
    assert torch.equal(torch.isnan(bad), hit)
    assert torch.equal(bad[~hit], got[~hit])


def test_training_products_of_one_layer():
    """y = x W', dx = dy W, dW = dy' x from the copies and transpose copies, each against the
    64-bit product of the values the copies stand for."""
    t, o, i = 70, 96, 130
    x, w, dy = rand((t, i), 1), rand((o, i), 2, sigma=0.05), rand((t, o), 3, sigma=0.1)
    pairs = [(M.mxfp4_quantize(x), M.mxfp4_quantize(w), i),
             (M.mxfp4_quantize(dy), M.mxfp4_quantize(w, transpose=True), o),
             (M.mxfp4_quantize(dy, transpose=True), M.mxfp4_quantize(x, transpose=True), t)]
    for (p, q, k), shape in zip(pairs, ((t, o), (t, i), (o, i))):
        a, b = R.mx_values(p.codes, p.scales, k), R.mx_values(q.codes, q.scales, k)
        got = M.mxfp4_product(p, q, F32)
        assert tuple(got.shape) == shape
        assert ((got.double().cpu() - a @ b.t()).abs() <= product_bound(a, b, k)).all()


def test_mxfp4_refusals():
    x = rand((4, 40), 1)
    q = M.mxfp4_quantize(x)
    with pytest.raises(ValueError):
        M.mxfp4_quantize(x.t())
    with pytest.raises(ValueError):
        M.mxfp4_quantize(x.cpu())
    with pytest.raises(ValueError):
        M.mxfp4_quantize(x, out=M.MXFP4.empty(40, 4, DEV))
    with pytest.raises(ValueError):
        M.mxfp4_quantize(x.double())
    with pytest.raises(ValueError):
        M.mxfp4_product(q, M.mxfp4_quantize(rand((4, 41), 1)))
    with pytest.raises(ValueError):
        M.mxfp4_product(q, q, out=torch.empty(4, 5, device=DEV))
    with pytest.raises(ValueError):
        M.mxfp4_dequantize(q, out=torch.empty(40, 4, device=DEV))
    with pytest.raises(ValueError):
        M.MXFP4(q.codes, q.scales, 4, 200)
    with pytest.raises(ValueError):
        M.MXFP4(q.codes.cpu(), q.scales, 4, 40)
    with pytest.raises(Z.NeoxError):
        M.mxfp4_quantize(x[:0])


# ----------------------------------------------------------------------------------------
# Muon
# ----------------------------------------------------------------------------------------

def weights(shapes, dtype, seed, scale=1024.0):
    out = []
    for i, s in enumerate(shapes):
        master = rand(s, seed + 10 * i, sigma=0.02)
        out.append(dict(grad=(rand(s, seed + 10 * i + 1, sigma=1e-4) * scale).to(dtype), half=master.to(dtype),
                        master=master, momentum=rand(s, seed + 10 * i + 2, sigma=3e-4), decay=i % 2 == 0))
    return out


def copy_of(ws):
    return [{k: v.clone() if hasattr(v, "clone") else v for k, v in w.items()} for w in ws]


def zcfg(dtype, **over):
    base = dict(beta1=0.95, weight_decay=0.1, clip_norm=1.0, init_scale=1024.0,
                dtype=Z.NEOX_F16 if dtype == F16 else Z.NEOX_BF16)
    base.update(over)
    return Z.neox_zero1_default_config(**base)


def check_step(before, after, state, cfg, lr, nesterov=1, mode="rms", ns=None):
    """One applied step against 64 bits.  The gradient factor is the library's own (unscale and
    clip coefficient as reported), so each tolerance counts only this element's roundings."""
    inv = cfg.predivide_factor / (cfg.dp_world_size * before["scale"])
    u = 2.0 ** -24
    for b, a in zip(before["w"], after):
        rows, cols = b["master"].shape
        mu = float(torch.tensor(cfg.beta1, dtype=F32))
        g = b["grad"].double().cpu() * (inv * state.last_clip_coef)
        m0 = b["momentum"].double().cpu()
        m = mu * m0 + g
        # g: factor rounded to FP32 (its two parts and their product), times the gradient; then
        # one fused multiply-add
        gerr = 4 * u * g.abs()
        merr = gerr + u * m.abs() + 2.0 ** -149
        assert ((a["momentum"].double().cpu() - m).abs() <= merr).all()
        # the direction from the stored momentum, as the kernels form it
        ms = a["momentum"].double().cpu()
        d = (g + mu * ms if nesterov else ms).float()
        kw = {} if ns is None else ns
        want, r, top = R.orth_bounds(d, F32, **kw)
        s = R.muon_scale(rows, cols, mode)
        lr32, wd = float(torch.tensor(lr, dtype=F32)), float(torch.tensor(cfg.weight_decay, dtype=F32))
        w0 = b["master"].double().cpu()
        dec = wd * w0 if b["decay"] else 0 * w0
        w = w0 - lr32 * (s * want + dec)
        werr = (a["master"].double().cpu() - w).abs()
        fl = 4 * u * (lr32 * (s * want.abs() + dec.abs()) + w.abs()) + 2.0 ** -149
        assert (werr <= lr32 * s * top + fl).all(), float((werr / (lr32 * s * top + fl)).max())
        assert R.rms(werr) <= lr32 * s * r + R.rms(fl), (R.rms(werr), lr32 * s * r, R.rms(fl))
        assert torch.equal(a["half"], a["master"].to(a["half"].dtype))
        assert torch.equal(a["grad"], b["grad"])


SETS = [[(64, 64)], [(1100, 530)], [(1, 1), (1, 5), (5, 1)], [(70, 33), (33, 70), (70, 33)], [(128, 384), (200, 130), (257, 129)]]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("shapes", SETS)
@pytest.mark.parametrize("nesterov,mode", [(1, "rms"), (0, "shape")])
def test_muon_step(dtype, shapes, nesterov, mode):
    cfg = zcfg(dtype)
    ws = weights(shapes, dtype, 100)
    mcfg = M.neox_muon_default_config(nesterov=nesterov, scale_mode=int(mode == "rms"))
    opt = M.Muon(cfg, [M.muon_matrix(**w) for w in ws], mcfg)
    for _ in range(2):
        st = opt.state()
        before = {"scale": st.loss_scale, "w": copy_of(ws)}
        opt.step(6e-4)
        st = opt.state()
        assert st.last_skipped == 0
        check_step(before, ws, st, cfg, 6e-4, nesterov, mode)
    assert st.step == 2


def test_muon_misaligned_arrays():
    """Arrays that start off any vector boundary."""
    cfg, ws = zcfg(BF16), weights([(37, 29), (64, 32)], BF16, 7)
    for w in ws:
        for k in ("grad", "half", "master", "momentum"):
            t = w[k]
            buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device=DEV)
            buf[1:] = t.reshape(-1)
            w[k] = buf[1:].view(t.shape)
    before = {"scale": 1024.0, "w": copy_of(ws)}
    opt = M.Muon(cfg, [M.muon_matrix(**w) for w in ws])
    opt.step(1e-3)
    check_step(before, ws, opt.state(), cfg, 1e-3)


def test_muon_scaler_matches_the_elementwise_step():
    """Scale, counters, norm and clip of each step, an overflow among them, are those of
    neox_zero1_step on the same gradients, bit for bit; a skipped step writes nothing else."""
    cfg = zcfg(F16, growth_interval=2, clip_norm=0.01, dp_world_size=2, predivide_factor=2.0)
    ws = weights([(40, 50), (64, 100)], F16, 3)
    scfg = zcfg(F16, growth_interval=2, clip_norm=0.01, dp_world_size=2, predivide_factor=2.0,
                optimizer=Z.NEOX_OPT_SGD)
    sgd_ws = copy_of(ws)
    sgd = Z.Zero1(scfg, [Z.segment(w["grad"].view(-1), w["half"].view(-1), w["master"].view(-1),
                                   w["momentum"].view(-1), None, w["decay"]) for w in sgd_ws])
    opt = M.Muon(cfg, [M.muon_matrix(**w) for w in ws])
    for k in range(6):
        for w, v in zip(ws, sgd_ws):
            g = rand(w["grad"].shape, 50 + k, sigma=1e-4) * opt.state().loss_scale
            if k in (1, 4):
                g[3, 5] = math.inf if k == 1 else math.nan
            w["grad"].copy_(g)
            v["grad"].copy_(w["grad"])
        before = {"scale": opt.state().loss_scale, "w": copy_of(ws)}
        opt.step(1e-3)
        sgd.step(1e-3)
        a, b = opt.state(), sgd.state()
        for f in ("loss_scale", "good_steps", "step", "skipped_total", "consecutive_overflows", "last_skipped",
                  "last_grad_norm", "last_clip_coef", "last_sumsq"):
            assert getattr(a, f) == getattr(b, f), (k, f)
        assert a.last_skipped == (k in (1, 4))
        if a.last_skipped:
            for x, y in zip(ws, before["w"]):
                assert all(torch.equal(x[n], y[n]) for n in ("half", "master", "momentum"))
        else:
            check_step(before, ws, a, cfg, 1e-3)


@pytest.mark.parametrize("count,shape", [(1, (130, 140)), (3, (257, 300)), (260, (130, 129))],
                         ids=["one", "three", "many"])
def test_muon_decisions_of_larger_matrices(count, shape):
    """The same for matrices that take many launches each, from one to more than 256 partial norms
    (neox_zero1_step decides in its update up to there): scaler state as neox_zero1_step's,
    weights as the formulas', MXFP4 copies rewritten by applied steps only."""
    kw = dict(growth_interval=2, clip_norm=0.01)
    cfg, ws = zcfg(F16, **kw), weights([shape] * count, F16, 13)
    copies = [(M.MXFP4.empty(*shape, DEV), M.MXFP4.empty(*shape[::-1], DEV)) for _ in ws[:2]]
    for c, t in copies:
        for a in (c.codes, c.scales, t.codes, t.scales):
            a.fill_(77)
    sgd_ws = copy_of(ws)
    sgd = Z.Zero1(zcfg(F16, optimizer=Z.NEOX_OPT_SGD, **kw),
                  [Z.segment(w["grad"].view(-1), w["half"].view(-1), w["master"].view(-1),
                             w["momentum"].view(-1), None, w["decay"]) for w in sgd_ws])
    opt = M.Muon(cfg, [M.muon_matrix(**w, **(dict(copy=copies[i][0], copy_t=copies[i][1]) if i < 2 and i < len(copies) else {}))
                       for i, w in enumerate(ws)])
    for k in range(4):
        for i, (w, v) in enumerate(zip(ws, sgd_ws)):
            g = rand(shape, 100 * k + i, sigma=1e-4) * opt.state().loss_scale
            if k in (0, 2) and i == count - 1:
                g[-1, -1] = math.inf
            w["grad"].copy_(g)
            v["grad"].copy_(w["grad"])
        before = {"scale": opt.state().loss_scale, "w": copy_of(ws)}
        old = [[a.clone() for a in (c.codes, c.scales, t.codes, t.scales)] for c, t in copies]
        opt.step(1e-3)
        sgd.step(1e-3)
        a, b = opt.state(), sgd.state()
        for f in ("loss_scale", "good_steps", "step", "skipped_total", "consecutive_overflows", "last_skipped",
                  "last_grad_norm", "last_clip_coef", "last_sumsq"):
            assert getattr(a, f) == getattr(b, f), (k, f)
        assert a.last_skipped == (k in (0, 2))
        if a.last_skipped:
            for x, y in zip(ws, before["w"]):
                assert all(torch.equal(x[n], y[n]) for n in ("half", "master", "momentum"))
            for (c, t), o in zip(copies, old):
                assert all(torch.equal(x, y) for x, y in zip((c.codes, c.scales, t.codes, t.scales), o))
        else:
            some = [0, count - 1] if count > 1 else [0]
            check_step({"scale": before["scale"], "w": [before["w"][i] for i in some]}, [ws[i] for i in some], a, cfg, 1e-3)
            for (c, t), w in zip(copies, ws):
                codes, scales = R.mx_quantize(w["master"])
                assert torch.equal(c.codes.cpu(), codes) and torch.equal(c.scales.cpu(), scales)
                codes, scales = R.mx_quantize(w["master"].t())
                assert torch.equal(t.codes.cpu(), codes) and torch.equal(t.scales.cpu(), scales)


@pytest.mark.parametrize("shape", [(70, 2100), (2500, 130), (1300, 700), (1030, 2200)])
def test_muon_step_of_other_shapes(shape):
    """Few rows and many columns (shares of the sums), either side longer, two steps at a time."""
    cfg, ws = zcfg(BF16), weights([shape], BF16, 17)
    opt = M.Muon(cfg, [M.muon_matrix(**w) for w in ws])
    before = {"scale": opt.state().loss_scale, "w": copy_of(ws)}
    opt.step(1e-3)
    check_step(before, ws, opt.state(), cfg, 1e-3)


def test_muon_and_adamw_share_one_decision():
    """A model as it is trained: matrices in a Muon handle, the rest in an AdamW shard, one norm
    over both, a step that the rest's gradient overflows, MXFP4 copies of the new weights, and a
    product with them."""
    dtype = BF16
    ws = weights([(96, 160), (160, 96)], dtype, 9)
    copies = [(M.MXFP4.empty(*w["master"].shape, DEV), M.MXFP4.empty(*w["master"].shape[::-1], DEV)) for w in ws]
    n = 777
    rest = dict(grad=rand((n,), 1, dtype, 0.1), half=rand((n,), 2, dtype), master=rand((n,), 2),
                exp_avg=torch.zeros(n, device=DEV), exp_avg_sq=torch.zeros(n, device=DEV))
    cfg = zcfg(dtype, clip_norm=0.02)
    opt = M.Muon(cfg, [M.muon_matrix(**w, copy=c, copy_t=t) for w, (c, t) in zip(ws, copies)])
    adam = Z.Zero1(cfg, [Z.segment(*rest.values(), decay=False)])
    sums = torch.zeros(2, dtype=torch.float64, device=DEV)
    for k in range(3):
        if k == 1:
            keep = rest["grad"].clone()
            rest["grad"][700] = math.nan
        if k == 2:
            rest["grad"].copy_(keep)
        before = {"scale": opt.state().loss_scale, "w": copy_of(ws)}
        old = [(c.codes.clone(), t.scales.clone()) for c, t in copies]
        s = Z.current_stream_ptr()
        M.neox_muon_step_local(opt.handle, sums.data_ptr(), s)
        Z.neox_zero1_step_local(adam.handle, sums.data_ptr() + 8, s)
        M.neox_muon_step_apply(opt.handle, sums.data_ptr(), 1e-3, s, nranks=2)
        Z.neox_zero1_step_apply(adam.handle, sums.data_ptr(), 1e-3, s, nranks=2)
        a, b = opt.state(), adam.state()
        for f in ("loss_scale", "good_steps", "step", "skipped_total", "consecutive_overflows", "last_skipped",
                  "last_grad_norm", "last_clip_coef", "last_sumsq"):
            assert getattr(a, f) == getattr(b, f), (k, f)
        if k == 1:
            assert a.last_skipped == 1
            for w, v, (c, t), o in zip(ws, before["w"], copies, old):
                assert all(torch.equal(w[x], v[x]) for x in ("half", "master", "momentum"))
                assert torch.equal(c.codes, o[0]) and torch.equal(t.scales, o[1])
            continue
        norm = math.sqrt(float(sums.sum()))
        assert abs(a.last_clip_coef - min(1.0, 0.02 / norm)) <= 2.0 ** -23
        check_step(before, ws, a, cfg, 1e-3)
        for w, (c, t) in zip(ws, copies):
            for q, tr in ((c, False), (t, True)):
                want = M.mxfp4_quantize(w["master"], transpose=tr)
                assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
    x = rand((5, 160), 4, BF16)
    y = M.mxfp4_product(M.mxfp4_quantize(x), copies[0][0], F32)
    a, b = (R.mx_values(q.codes, q.scales, 160) for q in (M.mxfp4_quantize(x), copies[0][0]))
    assert ((y.double().cpu() - a @ b.t()).abs() <= product_bound(a, b, 160)).all()


def test_muon_split_equals_whole_and_workspace_cap_does_not_matter():
    cfg = zcfg(F16)
    ws = weights([(100, 140)] * 5 + [(140, 60)] * 2, F16, 5)
    sums = torch.zeros(1, dtype=torch.float64, device=DEV)
    got = []
    for cap, split in ((0, False), (1, False), (3 << 20, True)):
        mine = copy_of(ws)
        opt = M.Muon(cfg, [M.muon_matrix(**w) for w in mine], M.neox_muon_default_config(workspace_bytes=cap))
        for _ in range(2):
            if split:
                M.neox_muon_step_local(opt.handle, sums.data_ptr(), Z.current_stream_ptr())
                M.neox_muon_step_apply(opt.handle, sums.data_ptr(), 1e-3, Z.current_stream_ptr())
            else:
                opt.step(1e-3)
        assert opt.state().step == 2
        got.append(mine)
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert all(torch.equal(a[k], b[k]) for k in ("half", "master", "momentum"))


def test_muon_resume():
    """A handle created from another's state and arrays goes on with the same bits."""
    cfg = zcfg(F16, growth_interval=2)
    ws = weights([(50, 70)], F16, 8)
    opt = M.Muon(cfg, [M.muon_matrix(**w) for w in ws])
    opt.step(1e-3)
    st, other = opt.state(), copy_of(ws)
    again = M.Muon(zcfg(F16, growth_interval=2, init_scale=st.loss_scale, init_step=st.step,
                        init_skipped=st.skipped_total, init_good_steps=st.good_steps,
                        init_consecutive_overflows=st.consecutive_overflows),
                   [M.muon_matrix(**w) for w in other])
    third = copy_of(ws)
    reset = M.Muon(cfg, [M.muon_matrix(**w) for w in third])
    M.neox_muon_scaler_set(reset.handle, st.loss_scale, st.good_steps, st.step, st.skipped_total,
                           st.consecutive_overflows, Z.current_stream_ptr())
    for o in (opt, again, reset):
        o.step(1e-3)
    for x in (again, reset):
        assert x.state().loss_scale == opt.state().loss_scale == 2048.0
    for a, b, c in zip(ws, other, third):
        assert all(torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]) for k in ("half", "master", "momentum"))


# ----------------------------------------------------------------------------------------
# streams and graphs
# ----------------------------------------------------------------------------------------

def test_results_on_another_stream_and_in_two_at_once():
    x, y = rand((3, 200, 300), 1), rand((3, 200, 300), 2)
    want = M.orthogonalize(x), M.orthogonalize(y)
    q = M.mxfp4_quantize(x[0])
    pwant = M.mxfp4_product(q, q, F32)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        a = M.orthogonalize(x)
        p = M.mxfp4_product(M.mxfp4_quantize(x[0]), q, F32)
    with torch.cuda.stream(t):
        b = M.orthogonalize(y)
    torch.cuda.synchronize()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(p, pwant)


def test_graphs_replay_with_new_inputs():
    """Captured calls, replayed with eager work between the replays, each against the eager
    result on the inputs of that replay."""
    x = rand((2, 150, 260), 1)
    xs, q = x.clone(), M.MXFP4.empty(150, 260, DEV)
    out, prod = torch.empty_like(x), torch.empty(150, 150, device=DEV)
    work = lambda: (M.orthogonalize(xs, out=out), M.mxfp4_quantize(xs[0], out=q),  # noqa: E731
                    M.mxfp4_product(q, q, out=prod))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        work()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for k in range(4):
        xs.copy_(rand((2, 150, 260), 20 + k))
        want = M.orthogonalize(xs)
        qq = M.mxfp4_quantize(xs[0])
        pw = M.mxfp4_product(qq, qq, F32)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(q.codes, qq.codes) and torch.equal(prod, pw), k


def test_muon_graph_replays_like_eager_steps():
    cfg = zcfg(F16, growth_interval=2)
    ws = weights([(80, 120), (120, 50)], F16, 6)
    eager = copy_of(ws)
    a = M.Muon(cfg, [M.muon_matrix(**w) for w in ws])
    b = M.Muon(cfg, [M.muon_matrix(**w) for w in eager])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step(1e-3)
    for k in range(5):
        for w, v in zip(ws, eager):
            w["grad"].copy_(rand(w["grad"].shape, 60 + k, sigma=0.1))
            if k == 2:
                w["grad"][1, 1] = math.inf
            v["grad"].copy_(w["grad"])
        g.replay()
        b.step(1e-3)
        torch.cuda.synchronize()
        for w, v in zip(ws, eager):
            assert all(torch.equal(w[n], v[n]) for n in ("half", "master", "momentum")), k
        assert a.state().loss_scale == b.state().loss_scale and a.state().step == b.state().step
    assert a.state().skipped_total == 1
