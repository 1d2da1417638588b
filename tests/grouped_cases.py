"""Cases of the grouped products, and which kernel takes each: the
groups' sizes are given, since a tile works its rows as 32, 64 or all of them.
test_gpu_grouped_tiles.py runs them; test_grouped_launches.py holds the library to the
kernels named here, so that a changed rule does not leave one without a test."""
import numpy as np

# sizes of the groups; 64 rows a tile below 384 rows a group, 96 from there on
SMALL = (0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 2, 17, 500, 100)
LARGE = (1500, 31, 65, 160)
TWO = (2100, 290)
ONE = (2304,)

# name -> (kernel, act, sizes, places of no group, K, N, R); kernel: <type> and <gated> are filled
# in.  R: x's rows, chosen by the plan with repetitions; None: x's rows are the places, or in any order.
TILED = {
    "16 x 64": ("mx_grouped16_kernel<{dt}, 4, {gated}>", "16bit", SMALL, 40, 416, 1568, None),
    "16 x 64, one K-tile": ("mx_grouped16_kernel<{dt}, 4, {gated}>", "16bit", SMALL, 0, 32, 1632, 300),
    "16 x 64, whole K-tiles": ("mx_grouped16_kernel<{dt}, 4, {gated}>", "16bit", SMALL, 5, 384, 1792, 900),
    "16 x 96": ("mx_grouped16_kernel<{dt}, 6, {gated}>", "16bit", LARGE, 30, 160, 1568, None),
    "16 x 96, two K-tiles": ("mx_grouped16_kernel<{dt}, 6, {gated}>", "16bit", LARGE, 0, 256, 1760, 500),
    "16 x 96, five K-tiles": ("mx_grouped16_kernel<{dt}, 6, {gated}>", "16bit", TWO, 3, 608, 1376, 1500),
    "4 x 64": ("mx_grouped4_kernel<{dt}, 4, 2, 1, 4, {gated}>", "mxfp4", SMALL, 40, 416, 608, None),
    "4 x 64, by row": ("mx_grouped4_kernel<{dt}, 4, 2, 1, 4, {gated}>", "mxfp4", SMALL, 7, 672, 544, 500),
    "4 x 64, one block": ("mx_grouped4_kernel<{dt}, 4, 2, 1, 4, {gated}>", "mxfp4", SMALL, 0, 32, 640, 1000),
    "4 x 128": ("mx_grouped4_kernel<{dt}, 4, 6, 2, 2, {gated}>", "mxfp4", LARGE, 30, 416, 3296, None),
    "4 x 128, by row": ("mx_grouped4_kernel<{dt}, 4, 6, 2, 2, {gated}>", "mxfp4", LARGE, 9, 608, 3392, 400),
    "4 x 128, five K-tiles": ("mx_grouped4_kernel<{dt}, 4, 6, 2, 2, {gated}>", "mxfp4", LARGE, 0, 640, 3296, 1200),
    "4 x 256": ("mx_grouped4_kernel<{dt}, 8, 8, 2, 2, {gated}>", "mxfp4", TWO, 20, 288, 7296, None),
    "4 x 256, by row": ("mx_grouped4_kernel<{dt}, 8, 8, 2, 2, {gated}>", "mxfp4", TWO, 1, 672, 7232, 600),
    "4 x 256, whole tiles": ("mx_grouped4_kernel<{dt}, 8, 8, 2, 2, {gated}>", "mxfp4", ONE, 0, 512, 7424, 2304),
}
# few rows a group, so many columns that a workgroup takes four panels
SPARSE = (1, 0, 3, 40, 2, 16, 0, 17, 5, 33, 1, 1, 0, 2, 4, 32, 0, 1, 6, 2, 0, 0, 9, 1, 3, 2, 1, 0, 15, 1)
FEW = {
    "few": ("mx_grouped_few_kernel<{dt}, false, {gated}, 4>", "16bit", SPARSE, 4, 352, 1120, None),
    "few, repeated rows": ("mx_grouped_few_kernel<{dt}, false, {gated}, 4>", "16bit", SPARSE, 0, 640, 1184, 50),
    "few, quantised": ("mx_grouped_few_kernel<{dt}, true, {gated}, 4>", "mxfp4", SPARSE, 4, 352, 1120, None),
    "few, quantised, repeated rows": ("mx_grouped_few_kernel<{dt}, true, {gated}, 4>", "mxfp4", SPARSE, 1, 1184, 1120, 60),
}
TILED.update(FEW)
TYPES = {"fp16": 0, "bf16": 1}


def kernel(name, dtype, gated):
    return TILED[name][0].format(dt=TYPES[dtype], gated=str(gated).lower())


def places(name, rng):
    """(offsets, rows) of a case; rows None: in place."""
    _, _, sizes, none, _, _, R = TILED[name]
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    S = offsets[-1] + none
    return offsets, rng.permutation(S) if R is None else rng.integers(0, R, S)


def columns(rng, N, gated):
    """Some of W's rows, those at the ends among them; with its up rows for gated ones."""
    n = N // 2 if gated else N
    some = np.unique(np.concatenate([[0, 1, 15, 16, n - 17, n - 16, n - 1], rng.integers(0, n, 200)]))
    return some, np.concatenate([some, some + n]) if gated else some


# adapters, as test_gpu_grouped.LORAS: M, L, r, K, N, share of rows without one
LORAS = [(1100, 3, 32, 160, 136, 0.1), (1536, 4, 24, 96, 259, 0), (1024, 2, 32, 64, 1040, 0.3)]

# choices by group, as test_gpu_grouped.test_group_rows: T, k, groups; few choices of many groups
ROWS = [(1, 1, 1024), (600, 2, 700), (3000, 2, 512), (6144, 1, 1000), (6145, 1, 900), (1, 6, 511)]
