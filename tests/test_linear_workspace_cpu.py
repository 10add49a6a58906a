"""What the linear layer's workspace queries go by: sizes, strides, types and the addresses'
alignment, not by the addresses themselves (host only; fake addresses)."""
import itertools

import pytest

pytest.importorskip("torch")

import mixed_precision_zero_amd as Z
from mixed_precision_zero_amd import linear as L

GAP = 1 << 36
X, W, Y, DY, PRE, DX, DW, DB, WORK = ((i + 16) * GAP for i in range(9))
# square ones, whose operands can be one array; rows of whole 16 bytes and others
SHAPES = [(333, 333, 333, 333), (64, 64, 64, 64), (64, 64, 64, 67), (1, 1, 1, 1), (5, 5, 5, 8), (2048, 2048, 2048, 2049)]


def gradients(at, m, n, k, ld, half, act, dbias, parts="xw"):
    dy, x, w = at
    return L.neox_linear_grads(dy=dy, pre=PRE if act else None, x=x, w=w, dx=DX if "x" in parts else None,
                               dw=DW if "w" in parts else None, dbias=DB if dbias else None, dy_ld=ld, pre_ld=ld,
                               x_ld=ld, w_ld=ld, dx_ld=ld, dw_ld=ld, m=m, n=n, k=k, dtype=half, act=act)


def layer(at, m, n, k, ld, half):
    x, w = at
    a = L.neox_linear_args(x=x, w=w, y=Y, x_ld=ld, w_ld=ld, y_ld=ld, m=m, n=n, k=k, y_dtype=half)
    a.epi.dtype = half
    return a


@pytest.mark.parametrize("half", [Z.NEOX_F16, Z.NEOX_BF16])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("off", [0, 2, 8])
def test_equal_and_distinct_operands_need_the_same(shape, off, half):
    """x, w and dy by one address, two of them by one, and all apart."""
    for act, dbias, parts in itertools.product((0, 2), (False, True), ("xw", "x", "w")):
        sizes = set()
        for at in itertools.product((X, W, DY), repeat=3):
            a = gradients([p + off for p in at], *shape, half, act, dbias, parts)
            sizes.add(L.neox_linear_backward_workspace(a))
        assert len(sizes) == 1, (act, dbias, parts, sizes)
    one, two = (L.neox_linear_workspace(layer((X + off, p + off), *shape, half)) for p in (X, W))
    assert one == two


def test_a_workspace_serves_other_addresses():
    """The size that a query with one address for all gives is enough for a call with distinct ones,
    and no more than enough."""
    shape = (333, 333, 333, 333)
    need = L.neox_linear_backward_workspace(gradients((X, X, X), *shape, Z.NEOX_F16, 0, False))
    assert need == 3 * ((333 * 384 * 2 + 255) // 256 * 256)
    a = gradients((DY, X, W), *shape, Z.NEOX_F16, 0, False)
    with pytest.raises(Z.NeoxError) as e:
        L.neox_linear_backward(a, WORK, need - 1)
    assert e.value.code == Z.NEOX_EINVAL and f"{need} needed" in str(e.value)


def test_no_tokens_leave_accumulated_gradients_alone():
    """Nothing is added to them, so nothing is launched (there may be no device)."""
    for act, dbias, parts in itertools.product((0, 2), (False, True), ("xw", "w", "")):
        if not dbias and not parts:
            continue
        a = gradients((DY, X, W), 0, 40, 50, 64, Z.NEOX_F16, act, dbias, parts)
        a.accumulate = 1
        assert L.neox_linear_backward_workspace(a) == 0
        L.neox_linear_backward(a, 0, 0)
    for dtype in (Z.NEOX_F16, Z.NEOX_BF16, L.NEOX_F32):
        L.neox_dropout_backward(None, 0, None, 0, DB, 1, 0, 40, dtype, None)
