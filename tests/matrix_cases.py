"""Shapes of MXFP4 products by the kernel that takes them (m, n, k): at least two for each, over many
slabs of K, with whole and half last slabs, whole and partial groups of scales, and cut tiles."""

import math

# the kernels, numbered as MxKernel in csrc/matrix_internal.h
TILES64, TILES128, TILES256, STREAM1X4, STREAM1X16, STREAM2X16, STREAM4X16 = range(7)

PRODUCTS_BY_KERNEL = [
    (STREAM1X4, 1, 24576, 6144), (STREAM1X4, 4, 24571, 1500), (STREAM1X4, 12, 16400, 2200),
    (STREAM1X16, 1, 77, 16384), (STREAM1X16, 16, 4096, 1600),
    (STREAM2X16, 17, 301, 4500), (STREAM2X16, 32, 4096, 1500),
    (STREAM4X16, 33, 1003, 5000), (STREAM4X16, 36, 4096, 900),
    (TILES64, 65, 1024, 16384), (TILES64, 333, 4096, 1024), (TILES64, 12, 40000, 1600), (TILES64, 60, 9001, 2200),
    (TILES128, 700, 5000, 4096), (TILES128, 2501, 9002, 1600),
    (TILES256, 4200, 4300, 1600), (TILES256, 2048, 8192, 2300),
]


# ----------------------------------------------------------------------------------------
# matrices on which an orthogonalisation's accuracy is held to the header's figures
# ----------------------------------------------------------------------------------------

def source(kind, rows, cols):
    """kind: "gauss", "rank N" (Gaussian factors), "sign" (rank 1 of +-1), "grid N" (N x N blocks of
    equal Gaussian values), "ones N" (N diagonal blocks of ones, zeros elsewhere), "rows" (one 1 a
    row)."""
    import torch
    g = torch.Generator().manual_seed(rows + cols)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    name, *n = kind.split()
    n = int(n[0]) if n else 0
    if name == "gauss":
        return rn(rows, cols)
    if name == "rank":
        return rn(rows, n) @ rn(n, cols)
    if name == "sign":
        return rn(rows, 1).sign() * rn(1, cols).sign()
    if name == "grid":
        return rn(n, n).repeat_interleave(-(-rows // n), 0)[:rows].repeat_interleave(-(-cols // n), 1)[:, :cols].contiguous()
    x = torch.zeros(rows, cols)
    if name == "rows":
        x[torch.arange(rows), torch.randint(0, cols, (rows,), generator=g)] = 1.0
        return x
    for i in range(n):
        x[rows * i // n:rows * (i + 1) // n, cols * i // n:cols * (i + 1) // n] = 1.0
    return x


def stated_error(kind, rows, cols):
    """The header's figure for such a matrix, relative to the result's norm."""
    m, n = sorted((rows, cols))
    if kind == "gauss":
        return 8e-3 if m < 16 else 3e-3
    if kind.startswith("rank"):
        return 3e-3 if m > 256 else 0.2 / math.sqrt(m)
    return 5e-2 if m > 512 and n >= 2 * m else 3e-2


ACCURACY = [("gauss", 64, 64), ("gauss", 100, 300), ("gauss", 387, 1001), ("gauss", 530, 1100), ("gauss", 700, 700),
            ("rank 1", 64, 64), ("rank 1", 60, 250), ("rank 1", 120, 90), ("rank 1", 300, 280), ("rank 1", 1200, 560),
            ("rank 1", 3, 4), ("rank 1", 8, 8), ("rank 1", 20, 50), ("rank 4", 33, 64), ("rank 8", 64, 64), ("rank 8", 353, 353),
            ("rank 8", 530, 1100), ("gauss", 2, 2), ("gauss", 9, 300), ("gauss", 1, 7),
            ("ones 1", 530, 1100), ("ones 1", 700, 700), ("ones 1", 353, 353), ("ones 1", 64, 64),
            ("ones 4", 300, 300), ("ones 4", 119, 402), ("ones 4", 448, 1372), ("ones 4", 1100, 530), ("ones 16", 600, 1300),
            ("ones 12", 134, 134), ("sign", 530, 1100), ("sign", 353, 353), ("grid 5", 530, 1100), ("grid 16", 200, 1000),
            ("rows", 353, 353), ("rows", 700, 700)]
# too large for the plain form on the CPU
ACCURACY_LARGE = [("ones 27", 2403, 5913), ("ones 4", 1144, 544), ("gauss", 2400, 5900), ("sign", 1030, 2100)]
