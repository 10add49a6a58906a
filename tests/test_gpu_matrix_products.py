"""Every kernel of the MXFP4 product over many slabs of K, against results that are exact."""
import pytest

torch = pytest.importorskip("torch")

import matrix_reference as R  # noqa: E402
from matrix_cases import PRODUCTS_BY_KERNEL  # noqa: E402
from mixed_precision_zero_amd import matrix as M  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32 = torch.float32


def integers(rows, k, seed):
    """A copy of values of {0, +-1, +-2, +-4} in blocks of scales 1, 2, 4 and 8, and its values: every
    sum of products of two of them is an integer of at most 1024 k."""
    g = torch.Generator().manual_seed(seed)
    x = torch.tensor([0.0, 1.0, 2.0, 4.0, -1.0, -2.0, -4.0])[torch.randint(0, 7, (rows, k), generator=g)]
    x[:, ::32] = 4.0 - 8.0 * (torch.arange(0, k, 32) % 3 == 0)
    q = M.mxfp4_quantize(x.to(DEV))
    up = torch.randint(0, 4, (rows, -(-k // 32)), generator=g, dtype=torch.uint8)
    q.scales[:, :up.shape[1]] += up.to(DEV)
    return q, R.mx_values(q.codes, q.scales, k)


@pytest.mark.parametrize("kernel,m,n,k", PRODUCTS_BY_KERNEL)
def test_product_kernels_are_exact_on_integers(kernel, m, n, k):
    assert 1024 * k <= 1 << 24                   # exact in FP32, in any order
    (qx, x), (qw, w) = integers(m, k, m), integers(n, k, n + 1)
    want = x @ w.t()
    buf = torch.full((m, n + 3), 7.0, device=DEV)
    M.mxfp4_product(qx, qw, out=buf[:, :n])
    got = M.mxfp4_product(qx, qw, F32)
    assert torch.equal(got.cpu().double(), want)
    assert torch.equal(buf[:, :n], got) and (buf[:, n:] == 7.0).all()
    # one block of NaN in the last slab of K, in a row of each operand
    last = (k - 1) // 32
    qx.scales[m // 2, last] = 255
    qw.scales[n - 1, last] = 255
    bad = M.mxfp4_product(qx, qw, F32).cpu()
    hit = torch.zeros(m, n, dtype=torch.bool)
    hit[m // 2], hit[:, n - 1] = True, True
    assert torch.equal(torch.isnan(bad), hit) and torch.equal(bad[~hit].double(), want[~hit])


@pytest.mark.parametrize("kernel,m,n,k", PRODUCTS_BY_KERNEL[::2])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_product_kernels_round_once(kernel, m, n, k, dtype):
    """16-bit results are the exact sums, rounded."""
    (qx, x), (qw, w) = integers(m, k, m + 2), integers(n, k, n + 3)
    qx.scales.sub_(7)                            # FP16's range
    want = (x @ w.t() / 128).to(F32).to(dtype)   # exact in FP32: rounded once
    assert torch.isfinite(want).all()
    assert torch.equal(M.mxfp4_product(qx, qw, dtype).cpu(), want)
