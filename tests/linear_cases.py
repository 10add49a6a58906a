"""Shapes of products by the kernel and the shares of K that take them: (kernel, shares > 1, I, J, K),
I columns and J rows of the result; the kernels numbered as ProductKernel in csrc/linear_internal.h."""

TILES64, TILES128, TILES128_DEEP, TILES256 = range(4)

PRODUCTS = [
    (TILES64, False, 8, 8, 8), (TILES64, False, 1000, 1000, 1000), (TILES64, False, 130, 70, 200),
    (TILES64, True, 128, 128, 16384), (TILES64, True, 1024, 333, 4096), (TILES64, True, 6144, 3, 8200),
    (TILES128, False, 4096, 2048, 1024), (TILES128, False, 3000, 3001, 500), (TILES128, False, 8000, 700, 40),
    (TILES128, True, 8, 3000, 32768), (TILES128, True, 1500, 1000, 16384),
    (TILES128_DEEP, False, 2000, 2000, 2000), (TILES128_DEEP, False, 6144, 333, 500),
    (TILES128_DEEP, True, 100, 1200, 8000), (TILES128_DEEP, True, 1500, 333, 4000),
    (TILES256, False, 8000, 333, 40), (TILES256, False, 4200, 4300, 200), (TILES256, False, 4096, 4096, 1000),
]

# Gradients of both operands by what takes them, (kernel, m, n, k): None for two launches, else the
# tiles of the one.
PAIRS = [
    (None, 1, 1001, 999), (None, 333, 4096, 999), (None, 4096, 3001, 4096),
    (TILES64, 387, 1001, 999), (TILES64, 100, 512, 1024),
    (TILES128, 700, 1001, 4096), (TILES128, 2048, 4096, 1024),
    (TILES128_DEEP, 387, 1001, 4096), (TILES128_DEEP, 3000, 100, 999),
]
