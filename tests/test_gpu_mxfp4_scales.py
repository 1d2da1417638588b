"""Weights at the ends of their scales: where a panel's values just fit fp16 or
just do not, fp16 subnormals among the operands, bf16's smallest and largest
values.  Inputs are scaled so that results are normal numbers: a kernel that
lost those weights would be far outside the bounds."""
import numpy as np
import pytest

import mx_reference as R
from test_gpu_mxfp4 import check, on_gpu, random_weights, shifted, tiled
from test_gpu_mxfp4_paths import clear_case, some_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_msd_amd as W
    W.lib()
    return t


SHAPES = [  # one, two and four tiles of few rows; the tiled product's three tiles
    (3, 1056, 100), (20, 672, 72), (50, 1056, 130), (1860, 2080, 4096), (600, 2208, 6000), (130, 672, 260),
]
FP16_ENDS = [  # scales, x's power of two: all of the panel exact in fp16 (the lower end: fp16 subnormals); none; some
    (104, 108, 12), (106, 113, 10), (137, 141, -10), (96, 104, 13), (141, 146, -14), (100, 109, 12),
]


@pytest.mark.parametrize("act", ["16bit", "mxfp4"])
@pytest.mark.parametrize("low,high,power", FP16_ENDS)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_fp16_products(torch, act, low, high, power, M, K, N):
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(M + low)
    x, exact = on_gpu(torch, rng.standard_normal((M, K)) * 2.0 ** power, "fp16")
    codes, _ = random_weights(rng, (N, K), zero_blocks=0)
    scales = rng.integers(low, high, (N, K // 32)).astype(np.uint8)
    rows = some_rows(rng, M)
    e = exact[rows] if act == "16bit" else R.dequantize(*R.quantize(exact[rows]))
    want, bound = R.matmul(e, R.dequantize(codes, scales), "fp16")
    assert np.median(np.abs(want)) > 2.0 ** -13 and np.abs(want).max() < 60000
    assert np.median(bound / np.maximum(np.abs(want), 1e-300)) < 0.05
    y = W.wqbmm_mxfp4_matmul(x, tiled(torch, codes, scales), N, activations=act)
    check(y[torch.from_numpy(rows).cuda()], want, bound)


@pytest.mark.parametrize("act", ["16bit", "mxfp4"])
@pytest.mark.parametrize("low,high,power", [(0, 6, 60), (0, 2, 100), (246, 253, -70), (251, 253, -100)])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_bf16_products(torch, act, low, high, power, M, K, N):
    """Scales from 0 (0.5 * 2^-127 is a bf16 subnormal) to 252 (6 * 2^125)."""
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(M + low)
    x, exact = on_gpu(torch, rng.standard_normal((M, K)) * 2.0 ** power, "bf16")
    codes, _ = random_weights(rng, (N, K), zero_blocks=0)
    scales = rng.integers(low, high, (N, K // 32)).astype(np.uint8)
    rows = some_rows(rng, M)
    e = exact[rows] if act == "16bit" else R.dequantize(*R.quantize(exact[rows]))
    want, bound = R.matmul(e, R.dequantize(codes, scales), "bf16")
    assert np.median(bound / np.maximum(np.abs(want), 1e-300)) < 0.05 and np.abs(want).max() < 2.0 ** 120
    y = W.wqbmm_mxfp4_matmul(x, tiled(torch, codes, scales), N, activations=act)
    check(y[torch.from_numpy(rows).cuda()], want, bound)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_magnitudes_from_2_to_the_128_on_are_not_finite(torch, dtype, M, K, N):
    """Scales 253 and 254 hold them, fp32 does not: their column is infinite or NaN, the
    others are as ever, also where such a scale holds smaller values."""
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(M)
    x, exact = on_gpu(torch, rng.choice([-1.0, 1.0], (M, K)) * (2.0 ** -120 if dtype == "bf16" else 2.0 ** -24), dtype)
    codes, scales = random_weights(rng, (N, K))
    c = np.stack([codes & 15, codes >> 4], -1).reshape(N, K)
    big = [3, 21, N - 1]
    scales[big] = 253
    c[big] = rng.integers(2, 6, (3, K))                  # 1 ... 3 times 2^126, all of one sign
    c[21, 40] = 7                                        # 6 times 2^126
    codes = (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)
    y = W.wqbmm_mxfp4_matmul(x, tiled(torch, codes, scales), N).double().cpu().numpy()
    assert not np.isfinite(y[:, 21]).any()
    rows, others = some_rows(rng, M), np.setdiff1d(np.arange(N), [21])
    want, bound = R.matmul(exact[rows], R.dequantize(codes, scales)[others], dtype)
    top = 65504.0 if dtype == "fp16" else 2.0 ** 127
    got = y[rows][:, others]
    assert np.isinf(got[np.abs(want) > 1.01 * top]).all()
    fits = np.abs(want) + bound < top
    assert (np.abs(got - want) <= bound)[fits].all() and fits.sum() >= (N - 3) * len(rows)


@pytest.mark.parametrize("up,down", [(-10, 34), (18, -26), (-16, 46), (24, -38)])
@pytest.mark.parametrize("T,H,inter,E,k", [(1, 288, 96, 6, 2), (20, 160, 64, 4, 2), (64, 544, 96, 3, 2), (64, 1056, 64, 33, 2)])
def test_fp16_experts(torch, up, down, T, H, inter, E, k):
    """Gate and up weights at the ends of what fp16 holds exactly, and beyond them."""
    import weight_only_quantized_msd_amd as W
    x, xe, router, re, gu, dn = clear_case(torch, T, H, inter, E, k, "fp16", T + H)
    gu, dn = (gu[0], shifted(gu[1], up)), (dn[0], shifted(dn[1], down))
    want, bound, *_ = R.moe(xe, re, R.dequantize(*gu), R.dequantize(*dn), k, True, "fp16")
    assert np.median(np.abs(want)) > 2.0 ** -13 and np.abs(want).max() < 60000
    assert np.median(bound / np.maximum(np.abs(want), 1e-300)) < 0.1
    y, _, _ = W.wqbmm_mxfp4_moe(x, router, tiled(torch, *gu), tiled(torch, *dn), inter, k)
    check(y, want, bound)
