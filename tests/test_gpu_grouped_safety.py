"""The operators whose weights depend on the row on the GPU: what a plan holds is not
trusted with memory, and calls on several streams at once do not meet."""
import numpy as np
import pytest

import grouped_cases as C
from test_gpu_mxfp4 import random_weights, same, tiled, torch  # noqa: F401

pytestmark = pytest.mark.gpu
GUARD = 4096


def gpu(torch, a):  # noqa: F811
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def guarded(torch, rows, cols):  # noqa: F811
    """A matrix between two stretches of 7."""
    all_ = torch.full((rows * cols + 2 * GUARD,), 7.0, dtype=torch.bfloat16, device="cuda")
    return all_, all_[GUARD:-GUARD].view(rows, cols)


def unbroken(all_):
    return bool((all_[:GUARD] == 7.0).all()) and bool((all_[-GUARD:] == 7.0).all())


def any_offsets(rng, G, S):
    """Descending, repeated, negative and far ones."""
    yield np.sort(rng.integers(0, S + 1, G + 1))[::-1]
    yield np.zeros(G + 1)
    yield np.full(G + 1, S)
    yield rng.choice([-2 ** 31, -1, 0, S // 2, S, S + 1, 2 ** 31 - 1], G + 1)
    yield np.where(np.arange(G + 1) % 2 == 0, 0, S)              # every second group has all places


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("name", ["16 x 64", "16 x 96", "4 x 64", "4 x 64, by row", "4 x 128", "4 x 256", "few", "few, quantised"])
def test_any_offsets_stay_within_the_matrices(torch, name, gather):  # noqa: F811
    import weight_only_quantized_msd_amd as W
    _, act, sizes, none, K, N, R = C.TILED[name]
    rng = np.random.default_rng(1)
    G, S = len(sizes), sum(sizes) + none
    R = R if gather and R else S
    x = torch.randn(R, K, device="cuda").bfloat16()
    wt = tiled(torch, *random_weights(rng, (G, N, K)))
    rows = gpu(torch, rng.choice([-1, 0, R - 1, R, 2 ** 31 - 1, -2 ** 31], S)) if gather else None
    for offsets in any_offsets(rng, G, S):
        all_, y = guarded(torch, S, N)
        W.wqbmm_mxfp4_grouped_matmul(x, wt, gpu(torch, offsets), N, rows=rows, activations=act, y=y)
        assert unbroken(all_)
        if not offsets.any():
            assert (y == 7.0).all()                              # no group has a place


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("M,L,r", [(100, 7, 16), (1100, 5, 72)])
def test_any_plan_of_adapters_stays_within_the_matrices(torch, M, L, r, in_place):  # noqa: F811
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(2)
    K, N = 96, 136
    x, a, b = (torch.randn(*s, device="cuda").bfloat16() for s in ((M, K), (L, r, K), (L, N, r)))
    for offsets in any_offsets(rng, L, M):
        rows = gpu(torch, rng.choice([-1, 0, M - 1, M, 2 ** 31 - 1, -2 ** 31], M))
        all_, y = guarded(torch, M, N)
        base = y if in_place else torch.zeros_like(y)
        W.wqbmm_lora_matmul(x, a, b, gpu(torch, offsets), rows, base=base, y=y)
        assert unbroken(all_)
        assert (y[1:M - 1] == 7.0).all()                         # rows that stand in no plan


def test_any_slots_stay_within_the_matrices(torch):  # noqa: F811
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(3)
    T, k, H, S = 50, 5, 264, 30
    z, weights = torch.randn(S, H, device="cuda").bfloat16(), torch.full((T, k), float("nan"), device="cuda")
    all_, y = guarded(torch, T, H)
    W.wqbmm_moe_combine(z, gpu(torch, rng.choice([-1, S, 2 ** 31 - 1, -2 ** 31], (T, k))), weights, y=y)
    assert unbroken(all_) and (y == 0).all()


def test_streams_at_once(torch):  # noqa: F811
    """Calls that pass values through the workspace, on three streams without a wait between them."""
    import weight_only_quantized_msd_amd as W
    _, _, sizes, _, K, N, _ = C.TILED["4 x 64"]
    rng = np.random.default_rng(4)
    G, S, L, r = len(sizes), 1532, 6, 72
    wt = tiled(torch, *random_weights(rng, (G, N, K)))
    a, b = torch.randn(L, r, K, device="cuda").bfloat16(), torch.randn(L, N, r, device="cuda").bfloat16()
    inputs = [(torch.randn(S, K, device="cuda").bfloat16(), gpu(torch, rng.integers(-1, G, 70000)),
               gpu(torch, rng.integers(-1, L, S)), gpu(torch, rng.integers(0, G, S))) for _ in range(12)]

    def calls(x, many, adapters, groups):
        plan, mine = W.wqbmm_group_rows(groups, G), W.wqbmm_group_rows(adapters, L)
        y = W.wqbmm_mxfp4_grouped_matmul(x, wt, plan[0], N, rows=plan[1], activations="mxfp4")
        return [*W.wqbmm_group_rows(many, G), y, W.wqbmm_lora_matmul(x, a, b, mine[0], mine[1], base=y)]

    want = [calls(*i) for i in inputs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for j, i in enumerate(inputs):
            with torch.cuda.stream(streams[j % 3]):
                got.append(calls(*i))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for one, two in zip(want, got) for p, q in zip(one, two))
