"""How many bits the expert layer's intermediate values h keep between its two
products: pairs of rows of h that differ by a few parts in 2^14 are subtracted,
which leaves in y what a rounding of h to fewer than 24 bits would cost."""
import numpy as np
import pytest

import mx_reference as R
from test_gpu_mxfp4 import check, on_gpu, tiled

pytestmark = pytest.mark.gpu

HALF32 = 2.0 ** -24                                     # half a step of fp32


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_msd_amd as W
    W.lib()
    return t


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def routed(rng, T, H, E):
    """x [T][H] with expert e's logit in column 64 + e (1/8 apart), and the router."""
    x, router = np.zeros((T, H)), np.zeros((E, H))
    router[:, 64:64 + E] = np.eye(E)
    x[:, 64:64 + E] = rng.permuted(np.tile(np.arange(E) / 8 - E / 16, (T, 1)), axis=1)
    return x, router


SHAPES = [  # T, H, I, E, k: one token, few by themselves, staged and direct rows, two and four panels
    (1, 128, 96, 4, 1), (1, 128, 1056, 20, 3), (2, 128, 64, 16, 2), (64, 512, 96, 4, 1), (64, 512, 96, 4, 2),
    (20, 1024, 2080, 3, 1), (60, 1024, 2080, 3, 2), (64, 2048, 64, 16, 1), (64, 2048, 64, 40, 2), (40, 2048, 160, 3, 1),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,H,inter,E,k", SHAPES)
def test_differences_of_intermediate_values(torch, dtype, T, H, inter, E, k):
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(T + H + inter)
    x, router = routed(rng, T, H, E)
    x[:, 0] = rng.choice([0.75, 1.0, 1.25, 1.75, -1.0, -1.5], T)
    x[:, 32] = rng.choice([1.0, -1.0], T)
    # rows 2p and 2p + 1: the same gate; up rows 2^10 times 1 ... 6, and 2^-4 times a value that differs
    gate_up, scales = np.zeros((E, 2 * inter, H), np.uint8), np.full((E, 2 * inter, H // 32), 127, np.uint8)
    gate_up[:, :inter, 0] = np.repeat(rng.integers(1, 6, (E, inter // 2)), 2, -1)
    gate_up[:, inter:, 0] = np.repeat(rng.integers(2, 8, (E, inter // 2)), 2, -1)
    gate_up[:, inter:, 32] = rng.integers(0, 8, (E, inter)) | (np.arange(inter) % 2 << 3)
    scales[:, inter:, 0], scales[:, inter:, 1] = 127 + 10, 127 - 4
    # column n of y: pair n % (I / 2), once with each sign
    down = np.zeros((E, H, inter), np.uint8)
    n = np.arange(H)
    down[:, n, 2 * (n % (inter // 2))], down[:, n, 2 * (n % (inter // 2)) + 1] = 2, 2 | 8
    x, xe = on_gpu(torch, x, dtype)
    router, re = on_gpu(torch, router, dtype)
    y, ids, _ = W.wqbmm_mxfp4_moe(x, router, tiled(torch, pack(gate_up), scales),
                                  tiled(torch, pack(down), np.full((E, H, inter // 32), 127, np.uint8)), inter, k)
    want_ids, shares, gap, slack = R.route(xe, re, k, True)
    assert gap > 4 * slack and np.array_equal(ids.cpu().numpy(), want_ids)
    gu = R.dequantize(pack(gate_up), scales)
    want, err = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            g, u = np.split(gu[want_ids[t, j]] @ xe[t], 2)       # sums of two terms, exact in fp32
            h = g / (1 + np.exp(-g)) * u * shares[t, j]
            at = 2 * (n % (inter // 2))
            # silu and the weight are off alike in both rows of a pair; two products are rounded in each
            want[t] += h[at] - h[at + 1]
            err[t] += np.abs(h[at] - h[at + 1]) * (8 * R.STEP32 + 2 * slack * 1.01 + (E + 16) * R.STEP32)
            err[t] += 2.02 * HALF32 * (np.abs(h[at]) + np.abs(h[at + 1]))
    err += (k + 3) * R.STEP32 * np.abs(want) + k * HALF32 * err
    bound = R.rounded(want, err, dtype)
    assert np.median(bound / np.maximum(np.abs(want), 1e-30)) < 2.0 ** -5      # what 16 bits would not keep
    check(y, want, bound)


@pytest.mark.parametrize("T,H,inter,E,k", [(1, 128, 64, 4, 1), (64, 512, 64, 4, 1), (64, 2048, 64, 16, 1)])
def test_infinite_intermediate_values(torch, T, H, inter, E, k):
    """h of the two signs beyond fp32: y is infinite where all shares have one sign, else NaN."""
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(3)
    x, router = routed(rng, T, H, E)
    x[:, 0] = 4.0
    gate_up, scales = np.zeros((E, 2 * inter, H), np.uint8), np.full((E, 2 * inter, H // 32), 127, np.uint8)
    gate_up[:, :inter, 0], gate_up[:, inter:, 0] = 7, 7
    gate_up[:, 2 * inter - 1, 0] = 7 | 8                          # the last row's h is -inf
    scales[:, :, 0] = 127 + 64
    down = rng.integers(1, 8, (E, H, inter)).astype(np.uint8)
    down[:, 1::4] |= 8                                            # all negative
    down[:, :, -1] ^= 8                                           # so that all shares have one sign
    down[:, 2::4, 5] ^= 8                                         # but for these columns
    x, router = on_gpu(torch, x, "bf16")[0], on_gpu(torch, router, "bf16")[0]
    y, _, _ = W.wqbmm_mxfp4_moe(x, router, tiled(torch, pack(gate_up), scales),
                                tiled(torch, pack(down), np.full((E, H, inter // 32), 127, np.uint8)), inter, k)
    y = y.float().cpu().numpy()
    assert (y[:, 0::4] == np.inf).all() and (y[:, 1::4] == -np.inf).all() and (y[:, 3::4] == np.inf).all()
    assert np.isnan(y[:, 2::4]).all()
