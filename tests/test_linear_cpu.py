"""The linear layer's C ABI without a GPU: symbols, structs, workspaces, every refusal
(arguments are checked before any device call, so fake addresses reach them), the kernels'
assembly, and the reference the GPU tests compare with."""
import ctypes as C
import math
import os
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")

import linear_reference as R
import mixed_precision_zero_amd as Z
from mixed_precision_zero_amd import build
from mixed_precision_zero_amd import linear as L
from linear_cases import PAIRS, PRODUCTS
from test_kernel_asm_cpu import PACKED_FP32, SCALAR_OK, _device_asm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GAP = 1 << 36
X, W, Y, B, RES, PRE, DY, DX, DW, DB, WORK, CNT = ((i + 16) * GAP for i in range(12))


def test_header_and_binding_agree():
    text = open(os.path.join(ROOT, "include", "neox_linear.h")).read()
    syms = sorted(set(re.findall(r"^int\s+(neox_\w+)\s*\(", text, re.M)))
    assert sorted(L.EXPORTS) == syms and len(syms) == 8
    for s in syms:
        assert hasattr(L.lib(), s)
    acts = dict(re.findall(r"^#define\s+NEOX_ACT_(\w+)\s+(\d)", text, re.M))
    assert {k.lower(): int(v) for k, v in acts.items()} == L.ACTS


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "neox_linear.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu %zu %zu", '
                   "sizeof(neox_drop), sizeof(neox_epilogue), sizeof(neox_linear_args), "
                   "sizeof(neox_linear_grads)); return 0; }\n")
    exe = str(tmp_path / "t")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe],
                   check=True)
    got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [C.sizeof(t) for t in (L.neox_drop, L.neox_epilogue, L.neox_linear_args,
                                                            L.neox_linear_grads)]


def refuses(text, f, *a, **k):
    with pytest.raises(Z.NeoxError) as e:
        f(*a, **k)
    assert e.value.code == Z.NEOX_EINVAL and text in str(e.value), str(e.value)


def forward(work=WORK, nbytes=1 << 34, dtype=Z.NEOX_BF16, act=0, bias=B, residual=RES, residual_ld=40, pre=PRE,
            pre_ld=40, p=0.1, counter=None, **kw):
    a = L.neox_linear_args(x=X, w=W, y=Y, x_ld=64, w_ld=64, y_ld=40, m=30, n=40, k=50, y_dtype=Z.NEOX_BF16)
    a.epi = L.neox_epilogue(dtype, act, bias, residual, residual_ld, pre, pre_ld, L.neox_drop(p, 1, 2, counter))
    for k, v in kw.items():
        setattr(a, k, v)
    return a, work, nbytes


def call_forward(**kw):
    a, work, nbytes = forward(**kw)
    L.neox_linear(a, work, nbytes)


FORWARD = [
    ("null", dict(x=None)), ("null", dict(w=None)), ("null", dict(y=None)),
    ("misaligned", dict(x=X + 1)), ("misaligned", dict(y=Y + 1)), ("misaligned", dict(bias=B + 1)),
    ("misaligned", dict(y=Y + 2, y_dtype=L.NEOX_F32)), ("misaligned", dict(counter=CNT + 4)),
    ("misaligned", dict(pre=PRE + 1)), ("misaligned", dict(residual=RES + 2, y_dtype=L.NEOX_F32)),
    ("not in [1", dict(n=0)), ("not in [1", dict(k=0)), ("not in [1", dict(n=(1 << 22) + 1)),
    ("not in [1", dict(k=(1 << 22) + 1, x_ld=1 << 23)), ("above 2^24", dict(m=(1 << 24) + 1)),
    ("tiles", dict(m=1 << 24, n=1 << 13)), ("type", dict(dtype=0)), ("type", dict(dtype=L.NEOX_F32)),
    ("y of type", dict(y_dtype=Z.NEOX_F16)), ("y of type", dict(y_dtype=9)), ("act", dict(act=5)),
    ("act", dict(act=-1)), ("reserved", dict(reserved=1)), ("p ", dict(p=-0.1)), ("p ", dict(p=1.1)),
    ("p ", dict(p=math.nan)), ("smaller", dict(x_ld=49)), ("smaller", dict(w_ld=49)), ("smaller", dict(y_ld=39)),
    ("smaller", dict(residual_ld=39)), ("smaller", dict(pre_ld=39)), ("above 2^40", dict(x_ld=1 << 41)),
    ("y meets x", dict(y=X)), ("y meets w", dict(y=W + 64)), ("y meets bias", dict(y=B - 200)),
    ("meets the residual", dict(residual=Y + 2)), ("meets the residual", dict(residual=Y, residual_ld=41)),
    ("meets y", dict(pre=Y)), ("pre meets x", dict(pre=X + 10)), ("pre meets the residual", dict(pre=RES)),
    ("y meets the counter", dict(counter=Y)), ("y meets x", dict(y=X, y_ld=64)),
]


@pytest.mark.parametrize("text,kw", FORWARD)
def test_linear_refuses(text, kw):
    refuses(text, call_forward, **kw)
    if "work" not in kw and "nbytes" not in kw:
        a, _, _ = forward(**kw)
        refuses(text, L.neox_linear_workspace, a)


def test_matrices_side_by_side_are_apart():
    """Columns of one wide array, as slices of a fused buffer are."""
    a, _, _ = forward(x=X, x_ld=200, y=X + 100, y_ld=200)              # columns 0..49 and 50..89
    L.neox_linear_workspace(a)
    a, _, _ = forward(x=X + 200, x_ld=200, y=X + 2 * 160, y_ld=200)    # 100..149 and 160..199
    L.neox_linear_workspace(a)
    a, _, _ = forward(x=X + 2 * 160, x_ld=210, y=X + 2 * 120, y_ld=210)
    L.neox_linear_workspace(a)
    refuses("y meets x", call_forward, x=X, x_ld=200, y=X + 98, y_ld=200)
    refuses("y meets x", call_forward, x=X, x_ld=200, y=X + 2 * 161, y_ld=200)
    refuses("y meets x", call_forward, x=X + 2 * 150, x_ld=200, y=X + 2 * 165, y_ld=200)
    refuses("y meets x", call_forward, x=X, x_ld=200, y=X + 100, y_ld=202)


def grads(work=WORK, nbytes=1 << 34, p=0.1, counter=None, **kw):
    a = L.neox_linear_grads(dy=DY, pre=PRE, x=X, w=W, dx=DX, dw=DW, dbias=DB, dy_ld=40, pre_ld=40, x_ld=64, w_ld=64,
                            dx_ld=50, dw_ld=50, m=30, n=40, k=50, dtype=Z.NEOX_F16, act=2)
    a.drop = L.neox_drop(p, 1, 2, counter)
    for k, v in kw.items():
        setattr(a, k, v)
    return a, work, nbytes


def call_backward(**kw):
    a, work, nbytes = grads(**kw)
    L.neox_linear_backward(a, work, nbytes)


@pytest.mark.parametrize("text,kw", [
    ("null", dict(dy=None)), ("null", dict(pre=None)), ("null", dict(x=None)), ("null", dict(w=None)),
    ("no gradient", dict(dx=None, dw=None, dbias=None)), ("type", dict(dtype=L.NEOX_F32)), ("act", dict(act=7)),
    ("accumulate", dict(accumulate=2)), ("reserved", dict(reserved=3)), ("p ", dict(p=2.0)),
    ("misaligned", dict(dy=DY + 1)), ("misaligned", dict(dw=DW + 1)), ("misaligned", dict(dbias=DB + 1)),
    ("smaller", dict(dx_ld=49)), ("smaller", dict(dy_ld=39)), ("smaller", dict(pre_ld=39)),
    ("not in [1", dict(k=0)), ("above 2^24", dict(m=1 << 25)), ("tiles", dict(n=1 << 22, k=1 << 21, dw_ld=1 << 21, w_ld=1 << 21, x_ld=1 << 21)),
    ("dx meets dy", dict(dx=DY)), ("dw meets w", dict(dw=W)), ("dbias meets dy", dict(dbias=DY + 8)),
    ("meets dx", dict(dw=DX)), ("meets dw", dict(dbias=DW + 20)), ("dx meets pre", dict(dx=PRE)),
    ("workspace", dict(work=None)), ("256-byte", dict(work=WORK + 64)), ("needed", dict(nbytes=100)),
    ("the workspace meets dy", dict(work=DY)), ("the workspace meets dw", dict(work=DW - 256)),
])
def test_linear_backward_refuses(text, kw):
    refuses(text, call_backward, **kw)


def mx(m=30, n=40, k=50, c=Y, dtype=Z.NEOX_BF16, ldc=40, half=Z.NEOX_BF16, act=0, p=0.0, bias=B, residual=None,
       codes=X, scales=X + GAP // 2, w=W, epi=True):
    e = L.neox_epilogue(half, act, bias, residual, 40, None, 0, L.neox_drop(p, 1, 2, None))
    if not epi:
        return Z._check(L.lib().neox_mxfp4_linear(codes, scales, m, w, w + GAP // 2, n, k, c, dtype, ldc, None, None))
    L.neox_mxfp4_linear(codes, scales, m, w, w + GAP // 2, n, k, c, dtype, ldc, e)


@pytest.mark.parametrize("text,kw", [
    ("null", dict(codes=None)), ("null", dict(scales=None)), ("null", dict(c=None)), ("null", dict(epi=False)),
    ("misaligned", dict(codes=X + 8)), ("misaligned", dict(scales=X + GAP // 2 + 2)), ("misaligned", dict(w=W + 4)),
    ("a product", dict(m=0)), ("a product", dict(n=0)), ("a product", dict(k=0)), ("a product", dict(k=(1 << 24) + 1)),
    ("a product", dict(m=1 << 31)), ("2^40", dict(m=1 << 20, k=1 << 24)), ("too large", dict(m=1 << 24, n=1 << 14, ldc=1 << 14)),
    ("type", dict(dtype=Z.NEOX_F16)), ("type", dict(half=7)), ("act", dict(act=9)), ("p ", dict(p=1.5)),
    ("smaller", dict(ldc=39)), ("meets a's codes", dict(c=X)), ("meets b's scales", dict(c=W + GAP // 2)),
    ("meets the residual", dict(residual=Y + 2)), ("meets bias", dict(bias=Y + 20)),
])
def test_mxfp4_linear_refuses(text, kw):
    refuses(text, mx, **kw)


def drop(x=X, x_ld=40, bias=B, residual=RES, residual_ld=40, y=Y, y_ld=40, rows=30, cols=40, dtype=Z.NEOX_F16,
         p=0.1, counter=None):
    L.neox_dropout(x, x_ld, bias, residual, residual_ld, y, y_ld, rows, cols, dtype, L.neox_drop(p, 1, 2, counter))


@pytest.mark.parametrize("text,kw", [
    ("null", dict(x=None)), ("null", dict(y=None)), ("type", dict(dtype=5)), ("a matrix", dict(cols=0)),
    ("a matrix", dict(rows=1 << 31)), ("smaller", dict(x_ld=39)), ("smaller", dict(y_ld=39)),
    ("smaller", dict(residual_ld=39)), ("misaligned", dict(x=X + 1)), ("misaligned", dict(bias=B + 2, dtype=L.NEOX_F32)),
    ("p ", dict(p=-1.0)), ("counter", dict(counter=CNT + 2)), ("y meets x", dict(y=X + 4)),
    ("y meets x", dict(y=X, y_ld=41)), ("y meets the residual", dict(y=RES + 2)), ("y meets bias", dict(y=B)),
])
def test_dropout_refuses(text, kw):
    refuses(text, drop, **kw)


def drop_back(dy=DY, dy_ld=40, dx=DX, dx_ld=40, dbias=DB, accumulate=0, rows=3000, cols=40, dtype=Z.NEOX_F16, p=0.1,
              work=WORK, nbytes=1 << 30):
    L.neox_dropout_backward(dy, dy_ld, dx, dx_ld, dbias, accumulate, rows, cols, dtype, L.neox_drop(p, 1, 2, None),
                            work, nbytes)


@pytest.mark.parametrize("text,kw", [
    ("null", dict(dy=None)), ("no gradient", dict(dx=None, dbias=None)), ("accumulate", dict(accumulate=-1)),
    ("type", dict(dtype=0)), ("a matrix", dict(cols=1 << 31)), ("smaller", dict(dx_ld=3)), ("smaller", dict(dy_ld=3)),
    ("p ", dict(p=math.inf)), ("dx meets dy", dict(dx=DY + 2)), ("dbias meets dy", dict(dbias=DY)),
    ("meets dx", dict(dbias=DX)), ("workspace", dict(work=None)), ("256-byte", dict(work=WORK + 2)),
    ("needed", dict(nbytes=1)), ("the workspace meets dy", dict(work=DY)),
])
def test_dropout_backward_refuses(text, kw):
    refuses(text, drop_back, **kw)


@pytest.mark.parametrize("rows,ld", [((1 << 20) + 2, 1 << 40), ((1 << 24) + 1, 1 << 40), ((1 << 25) + 1, 1 << 40),
                                     ((1 << 30) + 1, 1 << 34), ((1 << 31) - 1, 1 << 40)])
def test_spans_beyond_the_address_space_are_refused(rows, ld):
    """Also where rows times ld passes 64 bits."""
    for name in ("x", "residual", "y"):
        refuses(f"{name}: ld" if name != "residual" else "the residual: ld", drop, rows=rows, **{f"{name}_ld": ld})
    for name in ("dy", "dx"):
        refuses(f"{name}: ld", drop_back, rows=rows, **{f"{name}_ld": ld})
    if rows < 1 << 29:                      # (more have too many tiles)
        refuses("c: ld", mx, m=rows, ldc=ld)


def test_nothing_to_do_is_no_error():
    """No rows: nothing is read, written or launched."""
    L.neox_dropout(None, 0, None, None, 0, None, 0, 0, 40, Z.NEOX_F16, None)
    L.neox_dropout_backward(None, 0, None, 0, None, 0, 0, 40, Z.NEOX_F16, None)
    call_forward(m=0, x=None, y=None, residual=None, pre=None)
    a, _, _ = forward(m=0)
    assert L.neox_linear_workspace(a) == 0


def test_null_structs():
    n = C.c_uint64()
    f = L.lib()
    assert f.neox_linear(None, None, 0, None) == Z.NEOX_EINVAL
    assert f.neox_linear_workspace(None, C.byref(n)) == Z.NEOX_EINVAL
    assert f.neox_linear_workspace(C.byref(forward()[0]), None) == Z.NEOX_EINVAL
    assert f.neox_linear_backward(None, None, 0, None) == Z.NEOX_EINVAL
    assert f.neox_linear_backward_workspace(None, C.byref(n)) == Z.NEOX_EINVAL
    assert f.neox_linear_backward_workspace(C.byref(grads()[0]), None) == Z.NEOX_EINVAL
    assert f.neox_dropout_backward_workspace(3, 3, None) == Z.NEOX_EINVAL


def test_dropout_object_refuses():
    for kw in (dict(p=-0.1), dict(p=1.01), dict(p=math.nan), dict(p=0.1, seed=-1), dict(p=0.1, seed=1 << 64),
               dict(p=0.1, offset=1 << 64), dict(p=0.1, counter=torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            L.Dropout(**{"seed": 0, **kw})


def test_conveniences_refuse():
    x, w = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(6, 8, dtype=torch.float16)
    with pytest.raises(ValueError):
        L.linear(x, w)                                   # not on a GPU
    with pytest.raises(ValueError):
        L.linear(x.float(), w.float())
    with pytest.raises(ValueError):
        L.linear_backward(torch.zeros(4, 6, dtype=torch.float16), x, w)
    with pytest.raises(ValueError):
        L.dropout(x, None)
    with pytest.raises(ValueError):
        L.dropout_backward(x, None)


@pytest.mark.parametrize("src", [s for s in build.SOURCES if os.path.basename(s) in
                                 ("dropout_kernels.hip", "linear_kernels.hip")], ids=os.path.basename)
def test_kernel_assembly(src, tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    asm = _device_asm(src, tmp_path)
    n = len(re.findall(r"^\s*\.amdhsa_kernel\s+(\S+)", asm, re.M))
    assert n
    for field, want in ((r"\.amdhsa_float_denorm_mode_32", "3"), (r"\.amdhsa_float_denorm_mode_16_64", "3"),
                        (r"\.amdhsa_private_segment_fixed_size", "0")):
        assert re.findall(field + r"\s+(\d+)", asm) == [want] * n, field
    for field in ("vgpr_spill_count", "sgpr_spill_count"):
        got = re.findall(r"\." + field + r":\s+(\d+)", asm)
        assert len(got) == n and set(got) == {"0"}, (field, got)
    assert not re.search(r"^\s*scratch_", asm, re.M)
    assert not PACKED_FP32.search(asm)
    odd = sorted(m for m in set(re.findall(r"^\s+(s_[a-z0-9_]+)", asm, re.M)) if not m.startswith(SCALAR_OK))
    assert not odd, odd


# ----------------------------------------------------------------------------------------
# the reference itself
# ----------------------------------------------------------------------------------------

def test_philox_known_answers():
    """The three test vectors that come with the generator's publication."""
    f = 0xFFFFFFFF
    assert R.philox((0, 0, 0, 0), (0, 0)) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert R.philox((f, f, f, f), (f, f)) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert R.philox((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0)) == \
        [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def test_draws_are_philox():
    seed, off = 0x123456789ABCDEF0, 0xFEDCBA9876543210
    d = R.draws(seed, off, 5, 27)
    for r in range(5):
        for c in range(27):
            w = R.philox((c // 8, r, off & 0xFFFFFFFF, off >> 32), (seed & 0xFFFFFFFF, seed >> 32))[c % 8 // 2]
            assert int(d[r, c]) == (w >> 16 if c % 2 else w & 0xFFFF)


@pytest.mark.parametrize("name", R.ACTS)
def test_slopes_are_the_acts_derivatives(name):
    v = torch.linspace(-9, 9, 2001, dtype=torch.float64)
    v = v[v.abs() > 1e-3]
    h = 1e-5
    diff = (R.act(name, v + h) - R.act(name, v - h)) / (2 * h)
    assert float((diff - R.slope(name, v)).abs().max()) < 1e-8


def test_mask_follows_the_probability():
    """Counts of kept elements lie within five deviations of what p says."""
    for p in (0.1, 0.5, 0.9):
        scale, k = R.keep((p, 7, 11), 256, 1000)
        n, q = k.numel(), 1 - R.limit_of(p) / 65536
        assert abs(int(k.sum()) - n * q) < 5 * math.sqrt(n * q * (1 - q))
        assert abs(scale * q - 1) < 1e-7


# ----------------------------------------------------------------------------------------
# which kernel a product takes
# ----------------------------------------------------------------------------------------

class _Plan(C.Structure):
    _fields_ = [("kernel", C.c_int32), ("shares", C.c_uint32), ("slabs", C.c_uint64), ("cost", C.c_double)]


def plan(I, J, K):
    """The host's own choice (csrc/linear_internal.h)."""
    f = getattr(L.lib(), "_ZN3nz112product_planEmmm")
    f.argtypes, f.restype = [C.c_uint64] * 3, _Plan
    return f(I, J, K)


def test_every_product_kernel_has_its_shapes():
    """The list that the GPU tests run meets each kernel, with and without shares of K, twice or
    more, and a sweep of sizes takes none that the list leaves out."""
    got = [(plan(*s).kernel, plan(*s).shares > 1) for *_, I, J, K in PRODUCTS for s in [(I, J, K)]]
    assert got == [(kernel, shared) for kernel, shared, *_ in PRODUCTS]
    swept = set()
    for I in [1 << s for s in range(23)] + [1001, 3001, 24576]:
        for J in (0, 1, 7, 64, 100, 333, 1000, 2048, 3001, 8192, 65536):
            for K in (0, 1, 64, 1000, 6144, 16384, 1 << 22):
                if ((I + 63) // 64) * ((J + 63) // 64) <= 1 << 23:
                    p = plan(I, J, K)
                    swept.add((p.kernel, p.shares > 1))
                    # the shares cover K, none is empty, and the blocks fit a grid
                    slabs = max(1, -(-K // 64))
                    assert (p.shares - 1) * p.slabs < slabs <= p.shares * p.slabs
                    unit, threads = {0: (64, 256), 1: (128, 512), 2: (128, 512), 3: (128, 512)}[p.kernel]
                    assert -(-I // unit) * -(-J // unit) * p.shares * threads < 1 << 32
    assert swept == set(got) and all(got.count(k) > 1 for k in swept)


def pair(m, n, k):
    """Whether and how the host runs both gradients in one launch."""
    f = L.lib()["_ZN3nz19pair_planEmmRKNS_11ProductPlanEmmS2_PNS_13ProductKernelE"]
    U, P = C.c_uint64, C.POINTER(_Plan)
    f.argtypes, f.restype = [U, U, P, U, U, P, C.POINTER(C.c_int32)], C.c_bool
    x, w, kernel = plan(k, m, n), plan(k, n, m), C.c_int32()
    return kernel.value if f(k, m, C.byref(x), k, n, C.byref(w), C.byref(kernel)) else None


def test_every_pair_has_its_shapes():
    assert [pair(*s) for _, *s in PAIRS] == [kernel for kernel, *_ in PAIRS]
    swept = {pair(m, n, k) for m in (1, 64, 333, 1000, 2048, 5000) for n in (8, 512, 1001, 4096, 24576)
             for k in (8, 999, 1024, 6144)}
    assert swept == {kernel for kernel, *_ in PAIRS}


def test_workspaces_go_by_sizes_and_alignment():
    """Aligned operands need none but for shares; others room for their copies."""
    aligned = dict(x_ld=64, k=64, n=40)
    assert L.neox_linear_workspace(forward(**aligned)[0]) == 0
    one = L.neox_linear_workspace(forward(**dict(aligned, x=X + 2))[0])
    both = L.neox_linear_workspace(forward(**dict(aligned, x=X + 2, w=W + 2))[0])
    assert one == 30 * 64 * 2 and both == one + 40 * 64 * 2
    shared = dict(m=128, n=128, k=16384, x_ld=16384, w_ld=16384, y_ld=128, residual_ld=128, pre_ld=128)
    p = plan(128, 128, 16384)
    assert L.neox_linear_workspace(forward(**shared)[0]) == p.shares * 128 * 128 * 4
