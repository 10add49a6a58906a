"""Orthogonalisation against 64 bits, with the accuracy that include/neox_matrix.h states as the
limit, on matrices whose elements vary freely and on those where many are equal."""
import pytest

torch = pytest.importorskip("torch")

import matrix_reference as R  # noqa: E402
from matrix_cases import ACCURACY, ACCURACY_LARGE, source, stated_error  # noqa: E402
from mixed_precision_zero_amd import matrix as M  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def exact(x):
    """The polynomial in 64 bits on x's device."""
    if x.shape[0] > x.shape[1]:
        return exact(x.t().contiguous()).t()
    x = x.double()
    x = x / (torch.linalg.vector_norm(x) + 1e-7)
    for a, b, c in R.COEF:
        p = x @ x.t().contiguous()
        x = a * x + (b * p + c * (p @ p)) @ x
    return x


@pytest.mark.parametrize("kind,rows,cols", ACCURACY + ACCURACY_LARGE)
def test_stated_accuracy(kind, rows, cols):
    x = source(kind, rows, cols).to(DEV)
    got, want = M.orthogonalize(x).double(), exact(x)
    # FP32 results: their own rounding is 2^-24 of each element
    assert float((got - want).norm() / want.norm()) <= stated_error(kind, rows, cols) + 2.0 ** -24


@pytest.mark.parametrize("rows,cols", [(200, 300), (600, 1300)])
@pytest.mark.parametrize("tenths", [3, 5, 6])
def test_norms_far_below_eps(rows, cols, tenths):
    """Down to a norm of 1e-6 eps a matrix keeps the stated accuracy (results of about 5e-4 at most)."""
    x = source("gauss", rows, cols)
    x = (x * (1e-7 * 0.1 ** tenths / x.norm())).to(DEV)
    got, want = M.orthogonalize(x).double(), exact(x)
    assert float((got - want).norm() / want.norm()) <= stated_error("gauss", rows, cols) + 2.0 ** -24
