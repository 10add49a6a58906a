"""The linear layer's operators on the GPU where calls are unusual: operands that are one array,
no tokens."""
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
