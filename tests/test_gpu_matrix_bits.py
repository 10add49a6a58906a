"""What include/neox_matrix.h promises about bits: a matrix of a batch has the bits it has alone,
and neither workspace_bytes nor where the arrays lie changes a result."""
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_zero_amd as Z  # noqa: E402
from mixed_precision_zero_amd import matrix as M  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def rand(shape, seed, dtype=F32, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * sigma).to(dtype).to(DEV)


@pytest.mark.parametrize("count,rows,cols", [(8, 1024, 2100), (4, 700, 1500), (4, 1024, 4096), (5, 1300, 600),
                                             (40, 560, 1200), (9, 640, 700), (12, 200, 2500)])
def test_batches_have_the_bits_of_their_matrices(count, rows, cols):
    """Sizes whose launches take other tiles for a batch than for one matrix (two steps at a time,
    single steps, split sums); every matrix of the batch, and the batch again."""
    x = rand((count, rows, cols), 100 * count + rows, BF16)
    got = M.orthogonalize(x, dtype=F32)
    assert torch.equal(got, M.orthogonalize(x, dtype=F32))
    for i in range(count):
        assert torch.equal(got[i], M.orthogonalize(x[i], dtype=F32)), i


def test_equal_matrices_of_a_batch_are_equal():
    """The tiles of one launch differ from matrix to matrix: its last round is cut in quarters."""
    one = rand((1024, 2100), 3, BF16)
    got = M.orthogonalize(one.expand(8, 1024, 2100), out=torch.empty(8, 1024, 2100, device=DEV))
    assert all(torch.equal(got[0], got[i]) for i in range(1, 8))


def muon(ws, cfg, **over):
    return M.Muon(cfg, [M.muon_matrix(**w) for w in ws], M.neox_muon_default_config(**over))


@pytest.mark.parametrize("count,shape", [(8, (1024, 2100)), (5, (1300, 600))])
def test_muon_workspace_cap_keeps_the_bits(count, shape):
    cfg = Z.neox_zero1_default_config(beta1=0.95, weight_decay=0.1, init_scale=1024.0, dtype=Z.NEOX_BF16)
    got = []
    for cap in (0, 1):
        ws = []
        for i in range(count):
            w = rand(shape, 10 * i, sigma=0.02)
            ws.append(dict(grad=rand(shape, 10 * i + 1, BF16, 0.1), half=w.to(BF16), master=w,
                           momentum=rand(shape, 10 * i + 2, sigma=3e-4), decay=True))
        opt = muon(ws, cfg, workspace_bytes=cap)
        opt.step(1e-2)
        assert opt.state().last_skipped == 0
        got.append(ws)
    for a, b in zip(*got):
        assert all(torch.equal(a[k], b[k]) for k in ("half", "master", "momentum"))


# The next two tests look at X0 = source / (norm + eps) itself: one step of (a, b, c) = (1, 0, 0)
# gives it back.  Half of the source's elements are 1, and eps is swept over the doubles at which
# S / (norm + eps) passes a tie of FP32, 2^-5 (1 + 2^-24): there the last bit of the norm decides
# how all of them are rounded, so that another order of its sum shows.  S = 16 at 260 columns.
SIDE = 260
ULP = 2.0 ** -44                 # of norm + eps, just below 512


def ties(seed):
    x = rand((SIDE, SIDE), seed)
    x.view(-1)[::2] = 1.0
    return x


def swept(x):
    eps = 512.0 / (1 + 2.0 ** -24) - float(x.double().square().sum().sqrt())
    for k in range(-24, 25):
        yield M.neox_ns_default_config(coef=[(1.0, 0.0, 0.0)], eps=eps + k * ULP)


def off_by_one(t):
    """t's values in memory that starts one element behind a vector's boundary."""
    buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
    buf[1:] = t.reshape(-1)
    return buf[1:].view(t.shape)


@pytest.mark.parametrize("seed", range(6))
def test_norm_does_not_depend_on_strides_and_alignment(seed):
    x = ties(seed)
    wide = torch.zeros(SIDE, SIDE + 3, device=DEV)
    wide[:, :SIDE] = x
    odd = torch.zeros(2 * SIDE * SIDE + 1, device=DEV).as_strided((2, SIDE, SIDE), (SIDE * SIDE + 1, SIDE, 1))
    odd[0] = x
    ups = 0
    for cfg in swept(x):
        want = M.orthogonalize(x, cfg=cfg)
        ups += int((want.view(-1)[0] > 2.0 ** -9).item())
        assert torch.equal(M.orthogonalize(wide[:, :SIDE], cfg=cfg), want)
        assert torch.equal(M.orthogonalize(off_by_one(x), cfg=cfg), want)
        assert torch.equal(M.orthogonalize(odd, cfg=cfg)[0], want)
    assert 0 < ups < 49          # the sweep passed the tie


@pytest.mark.parametrize("seed", range(24))
def test_muon_norm_does_not_depend_on_alignment(seed):
    cfg = Z.neox_zero1_default_config(beta1=0.95, weight_decay=0.0, clip_norm=0.0, init_scale=1.0,
                                      scaler_mode=Z.NEOX_SCALER_STATIC, dtype=Z.NEOX_F16)
    m0 = rand((SIDE, SIDE), seed)
    m0.view(-1)[::2] = 0.0
    grad = torch.zeros(SIDE, SIDE, dtype=torch.float16, device=DEV)
    grad.view(-1)[::2] = 1.0
    ups = 0
    for ns in swept(m0 * 0.95 + grad.float()):
        got = []
        for place in (torch.clone, off_by_one):
            w = {k: place(t) for k, t in dict(grad=grad, half=grad * 0, master=m0 * 0, momentum=m0).items()}
            muon([dict(w, decay=False)], cfg, ns=ns, nesterov=0, scale_mode=M.NEOX_MUON_SCALE_SHAPE).step(1.0)
            got.append(w)
        torch.cuda.synchronize()
        ups += int((got[0]["master"].view(-1)[0] < -(2.0 ** -9)).item())
        assert all(torch.equal(got[0][k], got[1][k]) for k in ("master", "half", "momentum"))
    assert 0 < ups < 49
