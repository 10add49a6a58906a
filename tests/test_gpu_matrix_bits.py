"""What include/neox_matrix.h promises about bits: a matrix of a batch has the bits it has alone,
and neither workspace_bytes nor where the arrays lie changes a result."""
import math

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
