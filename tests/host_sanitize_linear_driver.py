"""Exercises the linear layer's host code (no GPU needed) for tests/test_sanitize_linear_cpu.py:
workspace queries over sizes, strides and alignments up to the limits, plans, the refusals of
every entry point, and calls up to their first launch, which has no device to go to.
Usage: python host_sanitize_linear_driver.py <path of the library build to load>."""
import itertools
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

import mixed_precision_zero_amd as Z  # noqa: E402

Z.LIB_PATH = sys.argv[1]
Z._lib = None
import test_linear_cpu as T  # noqa: E402
import test_linear_workspace_cpu as S  # noqa: E402
from mixed_precision_zero_amd import linear as L  # noqa: E402

launches = os.path.exists("/dev/kfd")        # (the addresses are made up: never launch on them)
queries = 0

# every operand aligned or not, rows of whole 16 bytes or not, no tokens, one, and the largest sides
SIDES = [(0, 5, 7), (0, 64, 64), (1, 1, 1), (1, 24576, 6144), (7, 1 << 22, 1), (3, 1, 1 << 22), (1 << 24, 8, 9),
         (1 << 24, 33, 64), (333, 1024, 4096), (387, 1001, 999), (2048, 4096, 1024), (8192, 24576, 6144), (64, 64, 16384)]
for (m, n, k), off, wide, half in itertools.product(SIDES, (0, 2), (0, 1, 1 << 22), (Z.NEOX_F16, Z.NEOX_BF16)):
    up = 1 << 38                             # the largest arrays are 2^24 rows of 2^23 elements
    at = [p + off for p in (up, 2 << 47, 3 << 47)]
    a = L.neox_linear_args(x=at[0], w=at[1], y=at[2], x_ld=k + wide, w_ld=k + wide, y_ld=n + wide, m=m, n=n, k=k,
                           y_dtype=half)
    a.epi = L.neox_epilogue(half, 2, 0, 0, 0, 0, 0, L.neox_drop(0.1, 1, 2, None))
    try:
        need = L.neox_linear_workspace(a)
        queries += 1
        if not launches:
            try:
                L.neox_linear(a, 7 << 47, need)
            except Z.NeoxError as e:
                assert e.code != Z.NEOX_EINVAL, e
    except Z.NeoxError as e:
        assert e.code == Z.NEOX_EINVAL, e
    for act, p, dbias, parts, acc in itertools.product((0, 3), (0.0, 0.2), (0, 6 << 47), ("xw", "x", "w", ""), (0, 1)):
        g = L.neox_linear_grads(dy=at[0], pre=at[1], x=at[2], w=(4 << 47) + off, dx=(5 << 47) if "x" in parts else 0,
                                dw=(8 << 47) if "w" in parts else 0, dbias=dbias, dy_ld=n + wide, pre_ld=n + wide,
                                x_ld=k + wide, w_ld=k + wide, dx_ld=k + wide, dw_ld=k + wide, m=m, n=n, k=k, dtype=half,
                                act=act, accumulate=acc)
        g.drop = L.neox_drop(p, 1, 2, None)
        try:
            need = L.neox_linear_backward_workspace(g)
            queries += 1
            if not launches:
                try:
                    L.neox_linear_backward(g, 7 << 47, need)
                except Z.NeoxError as e:
                    assert e.code != Z.NEOX_EINVAL, e
        except Z.NeoxError as e:
            assert e.code == Z.NEOX_EINVAL, e
assert queries > 1000, queries

for rows, cols in itertools.product((0, 1, 2, 1000, (1 << 31) - 1), (1, 7, 1037, 1 << 20, (1 << 31) - 1)):
    need = L.neox_dropout_backward_workspace(rows, cols)
    if not launches:
        for dtype in (Z.NEOX_F16, L.NEOX_F32):
            for call in (lambda: L.neox_dropout(1 << 47, cols, 0, 2 << 47, cols, 1 << 47, cols, rows, cols, dtype,
                                                L.neox_drop(0.5, 1, 2, None)) if rows < 1 << 20 or cols < 1 << 20 else None,
                         lambda: L.neox_dropout_backward(1 << 47, cols, 0, 0, 6 << 60, 0, rows, cols, dtype, None, 1 << 40, need)
                         if rows < 1 << 20 or cols < 1 << 20 else None):
                try:
                    call()
                except Z.NeoxError as e:
                    assert e.code != Z.NEOX_EINVAL, e
S.test_a_workspace_serves_other_addresses()
for shape in S.SHAPES:
    for off in (0, 2, 8):
        S.test_equal_and_distinct_operands_need_the_same(shape, off, Z.NEOX_BF16)


def table(f):
    """The cases that a test is parametrised by."""
    return [mark.args[1] for mark in f.pytestmark if mark.name == "parametrize"][0]


for test in (T.test_linear_refuses, T.test_linear_backward_refuses, T.test_mxfp4_linear_refuses, T.test_dropout_refuses,
             T.test_dropout_backward_refuses, T.test_spans_beyond_the_address_space_are_refused):
    for args in table(test):
        test(*args)
T.test_matrices_side_by_side_are_apart()
T.test_nothing_to_do_is_no_error()
T.test_null_structs()
T.test_every_product_kernel_has_its_shapes()
T.test_every_pair_has_its_shapes()
print("host code exercised", flush=True)
