"""The grouped products on the GPU, kernel by kernel, against the definition in 64 bits
(grouped_reference.py, which also derives the tolerances), a case for each kernel and
each way that it works a tile (grouped_cases.py)."""
import numpy as np
import pytest

import grouped_cases as C
import grouped_reference as G
import mx_reference as R
import test_gpu_grouped as V
from test_gpu_mxfp4 import check, on_gpu, random_weights, same, shifted, tiled, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def gpu(torch, a):  # noqa: F811
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def case(torch, name, dtype, seed):  # noqa: F811
    """x, its exact values, W's codes and scales, offsets, rows."""
    _, _, sizes, none, K, N, rows_of_x = C.TILED[name]
    rng = np.random.default_rng(seed)
    offsets, rows = C.places(name, rng)
    M = rows_of_x or len(rows)
    x, xe = on_gpu(torch, rng.standard_normal((M, K)) * 2.0 ** rng.integers(-2, 3, (M, 1)), dtype)
    return x, xe, random_weights(rng, (len(sizes), N, K)), offsets, rows, rng


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("name", C.TILED)
def test_tiles(torch, name, dtype, gated):  # noqa: F811
    import weight_only_quantized_msd_amd as W
    _, act, sizes, none, K, N, _ = C.TILED[name]
    x, xe, w, offsets, rows, rng = case(torch, name, dtype, K + N)
    some, of_w = C.columns(rng, N, gated)
    xq = R.dequantize(*R.quantize(xe)) if act == "mxfp4" else xe
    want, bound = G.grouped(xq, R.dequantize(w[0][:, of_w], w[1][:, of_w]), offsets, rows, gated, dtype)
    wt, off, o = tiled(torch, *w), gpu(torch, offsets), dict(activations=act, gated=gated)
    y = torch.full((len(rows), N // 2 if gated else N), 7.0, dtype=x.dtype, device="cuda")
    W.wqbmm_mxfp4_grouped_matmul(x, wt, off, N, rows=gpu(torch, rows), y=y, **o)
    n = offsets[-1]
    check(y[:n, torch.from_numpy(some).cuda()], want, bound)
    assert (y[n:] == 7.0).all()                                  # places of no group stay as they were
    # the same rows in their places, from a wider buffer
    wide = torch.full((len(rows) + 3, K + 72), float("nan"), dtype=x.dtype, device="cuda")
    wide[:len(rows), :K] = x[gpu(torch, rows).long()]
    there = W.wqbmm_mxfp4_grouped_matmul(wide[:len(rows), :K], wt, off, N, **o)
    assert same(torch, there[:n], y[:n])
    # all columns: W's rows in reverse give y's columns in reverse
    half = N // 2 if gated else N
    turn = np.arange(half)[::-1]
    whole = np.concatenate([turn, turn + half]) if gated else turn
    turned = tiled(torch, *(np.ascontiguousarray(t[:, whole]) for t in w))
    back = W.wqbmm_mxfp4_grouped_matmul(x, turned, off, N, rows=gpu(torch, rows), **o)
    assert same(torch, back[:n].flip(1).contiguous(), y[:n])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("name", ["16 x 64", "16 x 64, whole K-tiles", "16 x 96", "16 x 96, five K-tiles", "few"])
def test_weights_beyond_fp16(torch, name, gated):  # noqa: F811
    """fp16 x goes in two parts, 64 rows of a tile after the others, where some of its weights are beyond fp16."""
    import weight_only_quantized_msd_amd as W
    _, _, sizes, none, K, N, _ = C.TILED[name]
    x, xe, w, offsets, rows, rng = case(torch, name, "fp16", K)
    scales = w[1].copy()
    large = np.argsort(sizes)[-1]
    scales[large] = shifted(scales[large], -20)                  # all of a group, some rows of another
    scales[large - 1, 20:400] = shifted(scales[large - 1, 20:400], -25)
    some, of_w = C.columns(rng, N, gated)
    want, bound = G.grouped(xe, R.dequantize(w[0][:, of_w], scales[:, of_w]), offsets, rows, gated, "fp16")
    y = W.wqbmm_mxfp4_grouped_matmul(x, tiled(torch, w[0], scales), gpu(torch, offsets), N, rows=gpu(torch, rows), gated=gated)
    check(y[:offsets[-1], torch.from_numpy(some).cuda()], want, bound)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("name", C.TILED)
def test_nan_rows_and_rows_outside_x(torch, name, dtype):  # noqa: F811
    """A NaN or an infinity stays in its places, a row outside x gives zeros, and the others are as without them."""
    import weight_only_quantized_msd_amd as W
    _, act, sizes, none, K, N, _ = C.TILED[name]
    x, _, w, offsets, rows, rng = case(torch, name, dtype, K + N + 1)
    wt, off, o = tiled(torch, *w), gpu(torch, offsets), dict(activations=act, gated=True)
    clean = W.wqbmm_mxfp4_grouped_matmul(x, wt, off, N, rows=gpu(torch, rows), **o)
    n = offsets[-1]
    bad = rng.choice(rows[:n], 7, replace=False)
    x[torch.from_numpy(bad[:4]).cuda(), K - 3] = float("nan")
    x[torch.from_numpy(bad[4:]).cuda(), 5] = float("inf")
    moved = rows.copy()
    out = rng.choice(n, 9, replace=False)
    moved[out] = rng.choice([-1, -2 ** 31, len(x), 2 ** 31 - 1], 9)
    moved[n:] = 2 ** 31 - 1                                      # of no group: not looked at
    y = torch.full_like(clean, 7.0)
    W.wqbmm_mxfp4_grouped_matmul(x, wt, off, N, rows=gpu(torch, moved), y=y, **o)
    assert (y[n:] == 7.0).all()
    touched = np.isin(moved[:n], bad)
    gone = np.isin(np.arange(n), out)
    assert (y[:n][torch.from_numpy(gone).cuda()] == 0).all()
    assert torch.isnan(y[:n][torch.from_numpy(np.isin(moved[:n], bad[:4])).cuda()]).all()
    left = torch.from_numpy(~touched & ~gone).cuda()
    assert left.any() and same(torch, y[:n][left], clean[:n][left])


@pytest.mark.parametrize("name", ["16 x 64", "16 x 96", "4 x 64", "4 x 128, by row", "4 x 256"])
def test_replays(torch, name):  # noqa: F811
    """One captured call, with other rows, another order and other sizes of the groups each time."""
    import weight_only_quantized_msd_amd as W
    _, act, sizes, none, K, N, _ = C.TILED[name]
    x, _, w, offsets, rows, rng = case(torch, name, "bf16", 5)
    wt, off, at = tiled(torch, *w), gpu(torch, offsets), gpu(torch, rows)
    y = torch.zeros(len(rows), N // 2, dtype=x.dtype, device="cuda")

    def call(y):
        return W.wqbmm_mxfp4_grouped_matmul(x, wt, off, N, rows=at, activations=act, gated=True, y=y)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call(y)                                                  # the workspace grows before the capture
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call(y)
    for i in range(3):
        torch.cuda.synchronize()
        x.copy_(torch.randn_like(x))
        at.copy_(gpu(torch, rng.permutation(rows)))
        off.copy_(gpu(torch, np.concatenate([[0], np.cumsum(rng.permutation(sizes))])))
        y.fill_(i)
        want = call(torch.full_like(y, i))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        assert same(torch, y, want), i


# the further kernels that the cases of test_gpu_grouped.py do not reach
@pytest.mark.parametrize("T,k,groups", C.ROWS)
@pytest.mark.parametrize("kind", ["spread", "one", "in order", "any"])
def test_group_rows(torch, T, k, groups, kind):  # noqa: F811
    V.test_group_rows(torch, T, k, groups, kind)


@pytest.mark.parametrize("mixed", [True, False])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,L,r,K,N,none", C.LORAS)
def test_lora(torch, M, L, r, K, N, none, dtype, mixed):  # noqa: F811
    V.test_lora(torch, M, L, r, K, N, none, dtype, mixed)
