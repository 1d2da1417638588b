"""Products with 16-bit x whose last tile of rows is short, whose rows end inside
a K-tile, or both, for each workgroup tile; what stands around x is NaN."""
import numpy as np
import pytest

import mx_reference as R
from test_gpu_mxfp4 import check, on_gpu, random_weights, tiled
from test_gpu_mxfp4_paths import some_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_msd_amd as W
    W.lib()
    return t


@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N", [
    (1793, 4128, 4096), (1794, 4128, 4096), (1930, 2144, 4096),       # tiles of 128 rows: 1, 2 and 10 of the last
    (1860, 2080, 4096), (65, 4128, 4099), (449, 1056, 4096), (600, 2208, 6000),
])
def test_short_tiles_and_rows(torch, dtype, M, K, N, pad):
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(M + K + N)
    around = torch.full((M + 2, K + pad), float("nan"), dtype={"fp16": torch.float16, "bf16": torch.bfloat16}[dtype],
                        device="cuda")
    x, exact = on_gpu(torch, rng.standard_normal((M, K)), dtype)
    around[1:-1, :K] = x
    codes, scales = random_weights(rng, (N, K))
    w = tiled(torch, codes, scales)
    rows = np.union1d(some_rows(rng, M), np.arange(M // 64 * 64, M))
    y = W.wqbmm_mxfp4_matmul(around[1:-1, :K], w, N)
    assert not torch.isnan(y).any()
    check(y[torch.from_numpy(rows).cuda()], *R.matmul(exact[rows], R.dequantize(codes, scales), dtype))
