"""The launches of the operators whose weights depend on the row, without a GPU."""
import kernel_launches as K

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
