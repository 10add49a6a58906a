"""The matrix operators' C ABI without a GPU: symbols, defaults, sizes, and every refusal
(arguments are checked before any device call, so fake addresses reach them)."""
import ctypes as C
import math
import os
import re
import subprocess

import pytest

import mixed_precision_zero_amd as Z
from mixed_precision_zero_amd import build
from mixed_precision_zero_amd import matrix as M
from matrix_cases import ACCURACY, PRODUCTS_BY_KERNEL, source, stated_error
from test_kernel_asm_cpu import PACKED_FP32, SCALAR_OK, _device_asm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 40                      # fake device addresses, far apart
GAP = 1 << 36


def test_header_and_binding_agree():
    text = open(os.path.join(ROOT, "include", "neox_matrix.h")).read()
    syms = sorted(set(re.findall(r"^int\s+(neox_\w+)\s*\(", text, re.M)))
    assert sorted(M.EXPORTS) == syms and len(syms) == 15
    for s in syms:
        assert hasattr(M.lib(), s)


def test_header_is_plain_c(tmp_path):
    """The header compiles as C, and its structs have the binding's sizes."""
    src = tmp_path / "t.c"
    src.write_text('#include "neox_matrix.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu %zu", '
                   "sizeof(neox_ns_config), sizeof(neox_muon_config), sizeof(neox_muon_matrix)); return 0; }\n")
    exe = str(tmp_path / "t")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe],
                   check=True)
    got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [C.sizeof(t) for t in (M.neox_ns_config, M.neox_muon_config,
                                                            M.neox_muon_matrix)]


def test_defaults():
    c = M.neox_ns_default_config()
    assert c.steps == 5 and c.eps == 1e-7 and list(c.coef[4]) == [3.4445, -4.7750, 2.0315]
    c = M.neox_ns_default_config(coef=[(2.0, -1.5, 0.5), (1.5, -0.5, 0.0)])
    assert c.steps == 2 and list(c.coef[1]) == [1.5, -0.5, 0.0]
    m = M.neox_muon_default_config()
    assert (m.nesterov, m.scale_mode, m.workspace_bytes, m.ns.steps) == (1, M.NEOX_MUON_SCALE_RMS, 0, 5)
    with pytest.raises(AttributeError):
        M.neox_muon_default_config(momentum=0.9)
    with pytest.raises(ValueError):
        M.neox_ns_default_config(steps=3, coef=[(1.0, 0.0, 0.0)] * 2)


def refuses(text, f, *a, **k):
    with pytest.raises(Z.NeoxError) as e:
        f(*a, **k)
    assert e.value.code == Z.NEOX_EINVAL and text in str(e.value), str(e.value)


def orth(cfg=None, src=A, st=M.NEOX_F32, sld=40, ss=4000, dst=A + GAP, dt=M.NEOX_BF16, dld=40, ds=4000,
         count=2, rows=30, cols=40, scale=1.0, work=A + 2 * GAP, nbytes=None):
    M.neox_orthogonalize(cfg or M.neox_ns_default_config(), src, st, sld, ss, dst, dt, dld, ds, count, rows,
                         cols, scale, work, (1 << 30) if nbytes is None else nbytes)


@pytest.mark.parametrize("text,kw", [
    ("null", dict(src=None)), ("null", dict(dst=None)), ("null", dict(work=None)),
    ("types", dict(st=0)), ("types", dict(dt=4)), ("misaligned", dict(src=A + 2)),
    ("misaligned", dict(dst=A + GAP + 1)), ("256-byte", dict(work=A + 2 * GAP + 128)),
    ("needed", dict(nbytes=1000)), ("smaller than cols", dict(sld=39)), ("smaller than cols", dict(dld=39)),
    ("overlap", dict(ds=1199)), ("overlap", dict(dld=100, ds=39)), ("overlap", dict(dld=100, ds=61)),
    ("overlap", dict(dld=130, ds=60, count=3)), ("a matrix of", dict(rows=0)), ("a matrix of", dict(cols=0)),
    ("a matrix of", dict(rows=(1 << 20) + 1)), ("count", dict(count=0)), ("count", dict(count=(1 << 24) + 1)),
    ("scale", dict(scale=math.inf)), ("scale", dict(scale=math.nan)), ("scale", dict(scale=1e39)),
    ("overlaps src", dict(dst=A)), ("overlaps src", dict(dst=A, dt=M.NEOX_F32, ds=4001)),
    ("overlaps src", dict(dst=A + 4, dt=M.NEOX_F32)), ("workspace overlaps", dict(work=A)),
    ("workspace overlaps", dict(work=A + GAP - 256)), ("too large", dict(sld=1 << 60)),
    ("too large", dict(ss=1 << 62)),
])
def test_orthogonalize_refuses(text, kw):
    refuses(text, orth, **kw)


@pytest.mark.parametrize("text,change", [
    ("steps", dict(steps=0)), ("steps", dict(steps=17)), ("eps", dict(eps=0.0)), ("eps", dict(eps=math.nan)),
    ("eps", dict(eps=1e-60)), ("not finite", dict(coef=(math.inf, 0.0, 0.0))),
    ("grow", dict(coef=(9.0, 0.0, 0.0))), ("grow", dict(coef=(2.1, 0.0, 0.0))),
    ("too large", dict(coef=(1.0, 1e6, 0.0))), ("not finite", dict(coef=[(0.0, 0.0, 0.0), (1.0, 1e60, 0.0)])),
])
def test_orthogonalize_refuses_steps(text, change):
    refuses(text, orth, cfg=M.neox_ns_default_config(**change))


def test_reserved_and_null_configs():
    c = M.neox_ns_default_config()
    c.reserved = 1
    refuses("reserved", orth, cfg=c)
    L = M.lib()
    assert L.neox_ns_default_config(None) == Z.NEOX_EINVAL
    assert L.neox_muon_default_config(None) == Z.NEOX_EINVAL
    assert L.neox_orthogonalize(None, A, 3, 1, 1, A + GAP, 3, 1, 1, 1, 1, 1, 1.0, A + 2 * GAP, 1 << 30,
                                None) == Z.NEOX_EINVAL
    assert L.neox_orthogonalize_workspace(1, 1, 1, None) == Z.NEOX_EINVAL
    out = C.c_void_p()
    assert L.neox_muon_create(None, None, None, 1, None, C.byref(out)) == Z.NEOX_EINVAL
    assert L.neox_muon_step(None, 1.0, None) == Z.NEOX_EINVAL
    assert L.neox_muon_step_local(None, A, None) == Z.NEOX_EINVAL
    assert L.neox_muon_step_apply(None, A, 1, 1.0, None) == Z.NEOX_EINVAL
    assert L.neox_muon_state(None, None) == Z.NEOX_EINVAL
    assert L.neox_muon_scaler_set(None, None, None) == Z.NEOX_EINVAL
    assert L.neox_muon_destroy(None) == Z.NEOX_OK


def test_coefficients_that_stay_bounded_are_taken():
    """Known step polynomials pass the coefficients' check (the call stops at the workspace)."""
    for coef in ((3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0), (15 / 8, -10 / 8, 3 / 8), (2.0, -1.5, 0.5)):
        refuses("needed", orth, cfg=M.neox_ns_default_config(coef=coef), nbytes=0)


def test_matrices_side_by_side_are_taken():
    for kw in (dict(dld=100, ds=60), dict(dld=120, ds=40, count=3), dict(dld=40, ds=40, rows=1)):
        refuses("scale", orth, scale=math.inf, **kw)          # (the check behind those of the layout)


@pytest.mark.parametrize("count,rows,cols", [(1, 1, 1), (3, 1000, 37), (1, 1 << 20, 5), (64, 64, 64)])
def test_workspace_covers_the_iterate(count, rows, cols):
    n = M.neox_orthogonalize_workspace(count, rows, cols)
    m = min(rows, cols)
    assert n % 256 == 0 and n >= count * (8 * rows * cols + 4 * m * m)
    assert n <= count * (8 * (rows + 256) * (cols + 256) + 4 * (m + 256) ** 2 + 8 * (m + 256) + (1 << 13))


def mat(i=0, rows=8, cols=16, **over):
    base = A + 16 * i * GAP
    f = dict(grad=base, half=base + GAP, master=base + 2 * GAP, momentum=base + 3 * GAP, rows=rows, cols=cols,
             flags=0, reserved=0, mx_codes=None, mx_scales=None, mx_codes_t=None, mx_scales_t=None)
    f.update(over)
    return M.neox_muon_matrix(*f.values())


@pytest.mark.parametrize("text,mats,cfg,mcfg", [
    ("1 to 2^24", [], {}, {}),
    ("null array", [mat(grad=None)], {}, {}),
    ("null array", [mat(momentum=None)], {}, {}),
    ("a matrix of", [mat(rows=0)], {}, {}),
    ("a matrix of", [mat(cols=(1 << 20) + 1)], {}, {}),
    ("2-byte aligned", [mat(half=A + GAP + 1)], {}, {}),
    ("4-byte aligned", [mat(master=A + 2 * GAP + 2)], {}, {}),
    ("unknown flags", [mat(flags=2)], {}, {}),
    ("reserved", [mat(reserved=1)], {}, {}),
    ("written arrays overlap", [mat(0), mat(1, master=A + 2 * GAP + 256)], {}, {}),
    ("grad overlaps", [mat(grad=A + GAP)], {}, {}),
    ("half a pair", [mat(mx_codes=A + 8 * GAP)], {}, {}),
    ("half a pair", [mat(mx_scales_t=A + 8 * GAP)], {}, {}),
    ("misaligned", [mat(mx_codes=A + 8 * GAP + 8, mx_scales=A + 9 * GAP)], {}, {}),
    ("misaligned", [mat(mx_codes=A + 8 * GAP, mx_scales=A + 9 * GAP + 2)], {}, {}),
    ("copy overlaps", [mat(mx_codes=A + GAP, mx_scales=A + 9 * GAP)], {}, {}),
    ("copy overlaps", [mat(mx_codes=A + 8 * GAP, mx_scales=A)], {}, {}),
    ("copy overlaps", [mat(mx_codes=A + 8 * GAP, mx_scales=A + 9 * GAP, mx_codes_t=A + 8 * GAP + 64,
                           mx_scales_t=A + 10 * GAP)], {}, {}),
    ("beta1", [mat()], dict(beta1=1.0), {}),
    ("dtype", [mat()], dict(dtype=3), {}),
    ("optimizer", [mat()], dict(optimizer=2), {}),
    ("segment_norms", [mat()], dict(segment_norms=1), {}),
    ("init_scale", [mat()], dict(init_scale=0.0), {}),
    ("chunk_elems", [mat()], dict(chunk_elems=3), {}),
    ("nesterov", [mat()], {}, dict(nesterov=2)),
    ("scale_mode", [mat()], {}, dict(scale_mode=-1)),
    ("steps", [mat()], {}, dict(ns=M.neox_ns_default_config(steps=0))),
])
def test_muon_create_refuses(text, mats, cfg, mcfg):
    refuses(text, M.neox_muon_create, Z.neox_zero1_default_config(**cfg), M.neox_muon_default_config(**mcfg), mats)


def test_layout():
    assert M.neox_mxfp4_layout(1, 1) == (64, 4)
    assert M.neox_mxfp4_layout(7, 128) == (7 * 64, 7 * 4)
    assert M.neox_mxfp4_layout(7, 129) == (7 * 128, 7 * 8)
    for bad in ((0, 1), (1, 0), (1 << 31, 1), (1 << 30, 1 << 30)):
        refuses("copy of", M.neox_mxfp4_layout, *bad)
    assert M.lib().neox_mxfp4_layout(1, 1, None, None) == Z.NEOX_EINVAL


@pytest.mark.parametrize("text,a", [
    ("null", (None, 3, 8, 8, 8, 0, A, A + GAP)), ("null", (A, 3, 8, 8, 8, 0, None, A + GAP)),
    ("null", (A, 3, 8, 8, 8, 0, A + GAP, None)), ("type", (A, 0, 8, 8, 8, 0, A + GAP, A + 2 * GAP)),
    ("transpose", (A, 3, 8, 8, 8, 2, A + GAP, A + 2 * GAP)), ("ld", (A, 3, 8, 8, 7, 0, A + GAP, A + 2 * GAP)),
    ("copy of", (A, 3, 0, 8, 8, 0, A + GAP, A + 2 * GAP)), ("copy of", (A, 3, 8, 0, 8, 1, A + GAP, A + 2 * GAP)),
    ("misaligned", (A + 2, 3, 8, 8, 8, 0, A + GAP, A + 2 * GAP)),
    ("aligned", (A, 3, 8, 8, 8, 0, A + GAP + 8, A + 2 * GAP)),
    ("aligned", (A, 3, 8, 8, 8, 0, A + GAP, A + 2 * GAP + 1)),
    ("overlap", (A, 3, 8, 8, 8, 0, A + 128, A + 2 * GAP)), ("overlap", (A, 3, 8, 8, 8, 0, A + GAP, A + 252)),
    ("overlap", (A, 3, 8, 8, 8, 0, A + GAP, A + GAP + 508)),
])
def test_quantize_refuses(text, a):
    refuses(text, M.neox_mxfp4_quantize, *a)


@pytest.mark.parametrize("text,a", [
    ("null", (A, A + GAP, 8, 8, None, 3, 8)), ("null", (None, A + GAP, 8, 8, A + 2 * GAP, 3, 8)),
    ("type", (A, A + GAP, 8, 8, A + 2 * GAP, 5, 8)), ("ld", (A, A + GAP, 8, 8, A + 2 * GAP, 1, 7)),
    ("misaligned", (A, A + GAP, 8, 8, A + 2 * GAP + 1, 1, 8)), ("copy of", (A, A + GAP, 8, 0, A + 2 * GAP, 1, 8)),
    ("overlap", (A, A + GAP, 8, 8, A + 256, 1, 8)), ("overlap", (A, A + GAP, 8, 8, A + GAP + 16, 1, 8)),
])
def test_dequantize_refuses(text, a):
    refuses(text, M.neox_mxfp4_dequantize, *a)


@pytest.mark.parametrize("text,change", [
    ("null", {0: None}), ("null", {4: None}), ("null", {7: None}), ("copy of", {2: 0}), ("copy of", {5: 0}),
    ("copy of", {6: 0}), ("at most 2^24", {6: (1 << 24) + 1}), ("type", {8: 0}), ("ld", {9: 31}),
    ("misaligned", {7: A + 4 * GAP + 1}), ("aligned", {0: A + 4}), ("aligned", {4: A + 3 * GAP + 2}),
    ("overlaps", {7: A}), ("overlaps", {7: A + 3 * GAP}), ("too large", {2: 1 << 20, 5: 1 << 20, 9: 1 << 20}),
])
def test_product_refuses(text, change):
    a = [A, A + GAP, 16, A + 2 * GAP, A + 3 * GAP, 32, 100, A + 4 * GAP, M.NEOX_BF16, 32]
    for k, v in change.items():
        a[k] = v
    refuses(text, M.neox_mxfp4_product, *a)


@pytest.mark.parametrize("src", [s for s in build.SOURCES if os.path.basename(s) in
                                 ("matrix_kernels.hip", "mxfp4_kernels.hip")], ids=os.path.basename)
def test_kernel_assembly(src, tmp_path):
    """No scratch, no spills, no packed FP32, denormals kept, scalar memory only read."""
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    asm = _device_asm(src, tmp_path)
    n = len(re.findall(r"^\s*\.amdhsa_kernel\s+(\S+)", asm, re.M))
    assert n
    for field, want in ((r"\.amdhsa_float_denorm_mode_32", "3"), (r"\.amdhsa_float_denorm_mode_16_64", "3"),
                        (r"\.amdhsa_private_segment_fixed_size", "0")):
        assert re.findall(field + r"\s+(\d+)", asm) == [want] * n, field
    for field in ("vgpr_spill_count", "sgpr_spill_count"):
        assert set(re.findall(r"\." + field + r":\s+(\d+)", asm)) == {"0"}, field
    assert not re.search(r"^\s*scratch_", asm, re.M) and not PACKED_FP32.search(asm)
    odd = sorted(m for m in set(re.findall(r"^\s+(s_[a-z0-9_]+)", asm, re.M)) if not m.startswith(SCALAR_OK))
    assert not odd, odd


class OnDevice:
    """What muon_matrix asks of a tensor (or of an MXFP4 copy), on a device of the test's choice."""

    is_cuda = True

    def __init__(self, shape, dtype, device, at):
        self.shape, self.dtype, self.device, self.at = shape, dtype, device, at
        self.rows, self.cols = shape
        self._at = at, at + GAP

    def dim(self):
        return 2

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.at


@pytest.mark.parametrize("other", [None, "half", "master", "momentum", "copy", "copy_t"])
def test_muon_matrix_is_on_one_device(other):
    torch = pytest.importorskip("torch")
    kinds = dict(grad=torch.bfloat16, half=torch.bfloat16, master=torch.float32, momentum=torch.float32,
                 copy=None, copy_t=None)
    parts = {k: OnDevice((40, 24) if k == "copy_t" else (24, 40), dt, f"cuda:{int(k == other)}", A + 2 * i * GAP)
             for i, (k, dt) in enumerate(kinds.items())}
    if other is None:
        m = M.muon_matrix(**parts, decay=True)
        assert (m.grad, m.mx_codes, m.mx_scales_t, m.rows, m.cols) == (A, A + 8 * GAP, A + 11 * GAP, 24, 40)
        return
    with pytest.raises(ValueError, match="device"):
        M.muon_matrix(**parts, decay=True)


def product_kernel(m, n):
    """The host's own choice of a product's kernel (csrc/matrix_internal.h)."""
    f = getattr(M.lib(), "_ZN3nz117mx_product_kernelEmm")
    f.argtypes, f.restype = [C.c_uint64, C.c_uint64], C.c_int32
    return f(m, n)


def test_every_product_kernel_has_its_shapes():
    """The list that the GPU tests run meets each kernel twice or more, and a sweep of sizes takes no
    kernel that the list leaves out."""
    got = [product_kernel(m, n) for _, m, n, _ in PRODUCTS_BY_KERNEL]
    assert got == [kernel for kernel, *_ in PRODUCTS_BY_KERNEL]
    swept = {product_kernel(m, n) for m in list(range(1, 70)) + [100, 128, 333, 700, 2048, 8192, 60000]
             for n in [1 << s for s in range(22)] + [3 * 1001 ** 2 >> s for s in range(20)]}
    assert swept == set(got) and all(got.count(k) > 1 for k in swept)


@pytest.mark.parametrize("m", [1, 7, 16, 31, 64])
def test_streaming_products_fit_one_grid(m):
    """Blocks of 16 rows of b, up to 1,024 threads each, in fewer than 2^32 threads."""
    for n in [1 << s for s in range(31)] + [(1 << 29) + 1, 197149, 204800]:
        if product_kernel(m, n) >= 3:
            assert (n + 15) // 16 * 1024 < 1 << 32


@pytest.mark.parametrize("kind,rows,cols", ACCURACY)
def test_roundings_stay_within_the_stated_accuracy(kind, rows, cols):
    """The kernels' roundings alone, simulated, against the header's figures: what the GPU tests'
    tolerances are made of is itself held to a limit."""
    pytest.importorskip("torch")
    import matrix_reference as R
    x = source(kind, rows, cols)
    want = R.newton_schulz(x)
    err = R.newton_schulz_rounded(x) - want
    assert float(err.norm() / want.norm()) <= stated_error(kind, rows, cols)


def test_stated_accuracy_is_the_headers():
    text = " ".join(open(os.path.join(ROOT, "include", "neox_matrix.h")).read().split()).replace(" * ", " ")
    for words in ("as a rule, where G's elements vary freely; up to 3e-3, with a smaller side below 16 up to 8e-3",
                  "up to 0.2 / sqrt(smaller side) of the norm", "with a smaller side of up to 256, above that 3e-3 again",
                  "up to 3e-2 where many elements are equal", "4e-3 as a rule and up to 5e-2"):
        assert words in text, words
