"""The linear layer's operators on the GPU where calls are unusual: operands that are one array."""
import pytest

torch = pytest.importorskip("torch")

from mixed_precision_zero_amd import linear as L  # noqa: E402
from test_gpu_linear import HALVES, inside, ints, same_bits  # noqa: E402

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
