"""Shapes M, N, K of MXFP4 products by the kernel that they go to (a name of MxKernel in csrc/mx_index.h).

test_mx_index.py holds the rule to this table, test_mx_kernels_gpu.py compares each of its products with the oracle: a
limit of the rule that moves cannot leave a kernel untested."""

SHAPES = {
    # one slice of 128 channels, fewer slices than waves, whole rounds of the waves and a rest
    "Few2": [(1, 1, 128), (4, 1001, 640), (3, 70, 4096), (2, 333, 2176)],
    "Few4": [(1, 33, 4224), (4, 129, 14336), (3, 500, 8320)],
    # one stage, a part of one, several and a part; a tile's edges
    "Split": [(5, 40, 128), (33, 257, 640), (61, 130, 1152), (17, 96, 4224), (140, 260, 8320)],
    # stages fewer than the ring, odd and even; K beyond 4096 too
    "Tile64": [(640, 643, 128), (500, 1100, 384), (449, 1001, 512), (900, 904, 2176), (700, 1300, 896), (520, 1111, 4224)],
    "Tile128": [(1800, 2100, 128), (1801, 2096, 256), (1793, 2111, 384), (1920, 2048, 512), (1800, 2100, 1152),
                (3000, 1500, 640), (1795, 2077, 4224)],
    "Tile256": [(3841, 4096, 128), (3850, 4093, 256), (4096, 3588, 384), (3841, 3600, 512), (3900, 4001, 1152)],
}

ALL = [(kernel,) + shape for kernel, shapes in SHAPES.items() for shape in shapes]
