"""The launches of the operators whose weights depend on the row, without a GPU."""
import re

import grouped_cases as C
import kernel_launches as K
import test_gpu_grouped as V

# the ends of the sizes that include/wqbmm_grouped.h allows
LARGEST = (
    [K.route(2 ** 24, 1024, 16), K.group(2 ** 24, 1, 1024), K.group(1, 2 ** 24, 1)] +
    [K.combine(2 ** 24, 1024, 2 ** 14), K.combine(2 ** 18, 2, 2 ** 20), K.combine(2 ** 22, 1, 2 ** 13), K.combine(2 ** 24, 1, 8)] +
    [K.lora(M, L, r, 32, N) for M, N in ((2 ** 24, 2 ** 14), (2 ** 18, 2 ** 20), (2 ** 24, 1), (20000, 2 ** 20), (1000, 2 ** 20))
     for L in (1, 1024) for r in (8, 256)] +
    [K.grouped(S, G, k, N, act=act, gated=gated, R=R, ld=ld)
     for S, G, N in ((2 ** 24, 1024, 2 ** 14), (2 ** 24, 1, 2 ** 14), (2 ** 14, 1, 2 ** 24), (2 ** 17, 8, 2 ** 21), (2 ** 24, 3, 32),
                     (2 ** 18, 1024, 2 ** 14), (2 ** 16, 1024, 2 ** 14), (1, 1, 2 ** 24))
     for act in (0, 1) for gated in (0, 1)
     for k, R, ld in ((32, None, None), (32, 7, None), (32, None, 2 ** 23), (32, 1, 2 ** 36), (2 ** 20, 2 ** 24, None))])


def test_the_largest_sizes_fit_their_launches(tmp_path):
    """A launch holds fewer than 2^32 threads."""
    _, each = K.launched(tmp_path, LARGEST)
    few = set()
    for (name, args), (status, launches) in zip(LARGEST, each):
        assert status == 0 and launches, (name, args, status)
        assert all(0 < g * b < 2 ** 32 for _, g, b in launches), (name, args)
        if name == "wqbmm_moe_combine":
            T, H = args[7], args[4]
            assert sum(g * b for _, g, b in launches) >= T * H // 8, args
        if "grouped_few" in launches[0][0]:
            S, N, gated = args[7], args[9], args[13]
            wide = 32 if gated else 64                  # columns of a workgroup of four panels
            tiles = S // 32 + min(args[6], S)
            columns = N // (2 if gated else 1)
            assert sum(g for _, g, _ in launches) >= tiles * -(-columns // wide), args
            few.add(len(launches) > 1)
    assert few == {False, True}


def tiled_calls():
    for name, (_, act, sizes, none, k, N, R) in C.TILED.items():
        S = sum(sizes) + none
        for dtype, code in C.TYPES.items():
            for gated in (False, True):
                yield name, dtype, gated, K.grouped(S, len(sizes), k, N, code, int(act == "mxfp4"), int(gated), R or S)


def test_the_cases_reach_their_kernels(tmp_path):
    cases = list(tiled_calls())
    _, each = K.launched(tmp_path, [c[-1] for c in cases])
    for (name, dtype, gated, _), (status, launches) in zip(cases, each):
        assert status == 0 and launches[-1][0] == C.kernel(name, dtype, gated), (name, launches)


def calls_of_the_tests():
    """What the GPU tests of the values call, by its sizes."""
    for T, E, k in V.ROUTES:
        yield from (K.route(T, E, k, dtype) for dtype in (0, 1, 2))
    marks = {m.args[0]: m.args[1] for m in V.test_group_rows.pytestmark if m.name == "parametrize"}
    yield from (K.group(*sizes) for sizes in marks["T,k,groups"] + C.ROWS)
    for T, k, groups, Kx, N, _ in V.GROUPED:
        yield from (K.grouped(T * k, groups, Kx, N, dtype, act, gated, T)
                    for dtype in (0, 1) for act in (0, 1) for gated in (0, 1))
    for _, _, _, call in tiled_calls():
        yield call
    for M, L, r, Kx, N, _ in V.LORAS + C.LORAS:
        yield from (K.lora(M, L, r, Kx, N, dtype) for dtype in (0, 1))
    yield from (K.combine(96, 8, 2048, dtype) for dtype in (0, 1))


def test_every_kernel_is_reached_by_a_test(tmp_path):
    """Each instantiation that the library holds, by the cases of the tests that compare values on the GPU."""
    kernels, each = K.launched(tmp_path, list(calls_of_the_tests()))
    mine = {k for k in kernels if re.match(r"(route|group_rows|combine|lora_\w+|mx_grouped\w+|mx_row_codes)_kernel", k)}
    assert len(mine) > 60
    assert mine - {k for status, launches in each for k, _, _ in launches} == set()
