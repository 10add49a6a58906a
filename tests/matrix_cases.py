"""Shapes of MXFP4 products by the kernel that takes them (m, n, k): at least two for each, over many
slabs of K, with whole and half last slabs, whole and partial groups of scales, and cut tiles."""

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
