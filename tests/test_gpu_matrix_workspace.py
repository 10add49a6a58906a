"""The memory that the Newton-Schulz operators ask for, and what they do with it."""
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_zero_amd as Z  # noqa: E402
from mixed_precision_zero_amd import matrix as M  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rand(shape, seed, dtype=torch.float32, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * sigma).to(dtype).to(DEV)


@pytest.mark.parametrize("count,rows,cols", [(3, 64, 64), (2, 128, 100), (2, 40, 256), (2, 129, 60), (1, 300, 1000),
                                             (2, 60, 2100), (2, 560, 1200), (1, 1200, 560)])
def test_orthogonalize_stays_inside_its_workspace(count, rows, cols):
    need, guard = M.neox_orthogonalize_workspace(count, rows, cols), 1 << 16
    x, out = rand((count, rows, cols), rows), torch.empty(count, rows, cols, device=DEV)
    work = torch.full((need + guard,), 0xA5, dtype=torch.uint8, device=DEV)
    M.neox_orthogonalize(M.neox_ns_default_config(), x.data_ptr(), M.NEOX_F32, cols, rows * cols, out.data_ptr(),
                         M.NEOX_F32, cols, rows * cols, count, rows, cols, 1.0, work.data_ptr(), need,
                         Z.current_stream_ptr())
    assert torch.equal(out, M.orthogonalize(x))
    assert (work[need:] == 0xA5).all()
    lo, hi = sorted((rows, cols))
    if hi <= 128 or (lo <= 64 and hi <= 256):
        assert (work == 0xA5).all()              # one block does a matrix by itself


def test_muon_of_small_matrices_takes_no_workspace():
    """2,000 matrices that one block each does: what the handle allocates is its tables, not 50 KB a
    matrix, and workspace_bytes says nothing to it."""
    n, shape = 2000, (64, 64)
    grad, w = rand((n, *shape), 1, torch.bfloat16, 0.1), rand((n, *shape), 2, sigma=0.02)
    got = []
    for cap in (0, 1):
        half, master, mom = w.to(torch.bfloat16), w.clone(), torch.zeros_like(w)
        mats = [M.muon_matrix(grad[i], half[i], master[i], mom[i], decay=True) for i in range(n)]
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        opt = M.Muon(Z.neox_zero1_default_config(beta1=0.95, init_scale=1024.0, dtype=Z.NEOX_BF16), mats,
                     M.neox_muon_default_config(workspace_bytes=cap))
        assert before - torch.cuda.mem_get_info()[0] <= 16 << 20
        opt.step(1e-2)
        assert opt.state().step == 1
        got.append((half, master, mom))
        opt.close()
    assert all(torch.equal(a, b) for a, b in zip(*got))
