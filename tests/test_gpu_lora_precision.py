"""Low-rank adapters: how exactly B multiplies A.x, as include/wqbmm_grouped.h states it,
where the largest values of A.x meet zeros in B and the small ones make the result.  A.x
is one product of powers of two and a few bits, exact in fp32."""
import numpy as np
import pytest

from mx_reference import STEP32, rounded
from test_gpu_mxfp4 import on_gpu, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def run(torch, x, a, b, dtype):  # noqa: F811
    import weight_only_quantized_msd_amd as W
    (x, xe), (a, ae), (b, be) = (on_gpu(torch, t, dtype) for t in (x, a, b))
    ids = torch.zeros(len(x), dtype=torch.int32, device="cuda")
    offsets, rows, _ = W.wqbmm_group_rows(ids, 1)
    y = W.wqbmm_lora_matmul(x, a[None], b[None], offsets, rows).double().cpu().numpy()
    return y, xe @ ae.T, be


@pytest.mark.parametrize("M", [40, 1100])
@pytest.mark.parametrize("r", [16, 72])
def test_fp16_below_the_largest_of_a_row(torch, M, r):  # noqa: F811
    rng = np.random.default_rng(M + r)
    K, N = 64, 104
    x, a, b = np.zeros((M, K)), np.zeros((r, K)), rng.standard_normal((N, r))
    x[:, 0], x[:, 1] = 2.0 ** 10, 2.0 ** -10 * rng.integers(1, 2 ** 11, M) / 2 ** 10
    a[:8, 0] = rng.standard_normal(8)                            # the large ones
    a[8:, 1] = rng.standard_normal(r - 8) * 2.0 ** -rng.integers(0, 14, r - 8)
    b[:, :8] = 0
    y, v, b = run(torch, x, a, b, "fp16")
    top = np.abs(v).max(1, keepdims=True)
    small = np.abs(v[:, 8:])
    assert (small < 2.0 ** -16 * top).mean() > 0.9 and (small > 2.0 ** -38 * top).mean() > 0.5
    e = np.maximum(2.0 ** -22 * np.abs(v), 2.0 ** -38 * top) @ np.abs(b).T
    e += 2 * r * STEP32 * (np.abs(v) @ np.abs(b).T)
    want = v @ b.T
    assert (np.abs(y - want) <= rounded(want, e, "fp16")).all()


@pytest.mark.parametrize("M", [40, 1100])
@pytest.mark.parametrize("r", [16, 72])
def test_bf16_at_the_lower_end(torch, M, r):  # noqa: F811
    rng = np.random.default_rng(M + r)
    K, N = 64, 104
    x, a = np.zeros((M, K)), np.zeros((r, K))
    x[:, 1] = 2.0 ** -60 * rng.integers(2 ** 7, 2 ** 8, M)
    down = np.concatenate([rng.integers(45, 60, 8), rng.integers(80, 92, r - 8)])
    a[:, 1] = rng.choice([-1, 1], r) * 2.0 ** -down * rng.integers(2 ** 7, 2 ** 8, r)
    b = rng.standard_normal((N, r)) * 2.0 ** rng.integers(90, 120, (N, 1))
    b[:, :8] = 0
    y, v, b = run(torch, x, a, b, "bf16")
    assert np.abs(v).min() < 2.0 ** -133 and np.abs(v).max() > 2.0 ** -100
    e = np.where(np.abs(v) < 2.0 ** -110, 2.0 ** -133, 0.0) @ np.abs(b).T
    e += np.full_like(v, 2.0 ** -149) @ np.abs(b).T              # v itself in fp32
    e += 3 * r * STEP32 * (np.abs(v) @ np.abs(b).T)
    want = v @ b.T
    assert (np.abs(y - want) <= rounded(want, e, "bf16")).all()
