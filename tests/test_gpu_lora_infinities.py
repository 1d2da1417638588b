"""Low-rank adapters with infinities and NaN in B, A and x: the definition's values in 64
bits, infinite and NaN where it is.  A.x is multiplied in parts that each meet B, so
that a part of 0, or of the other sign, must not meet an infinity."""
import numpy as np
import pytest

import grouped_reference as G
from test_gpu_mxfp4 import on_gpu, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def definition(x, a, b, ids, scales, base):
    with np.errstate(invalid="ignore", over="ignore"):
        y = base.copy()
        for m, l in enumerate(ids):
            if l >= 0:
                v = (x[m] * a[l]).sum(1) * scales[l]
                y[m] += (v * b[l]).sum(1)
    return y


def finite(t):
    return np.where(np.isfinite(t), t, 0.0)


@pytest.mark.parametrize("values", ["whole", "any", "far"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,L,r,K,N", [(40, 3, 8, 64, 97), (33, 2, 72, 32, 264), (20, 2, 256, 96, 40), (1030, 2, 16, 64, 136),
                                       (1025, 1, 136, 32, 72)])
def test_infinities_are_followed(torch, M, L, r, K, N, dtype, values):  # noqa: F811
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(M + r + N)
    if values == "whole":                                        # A.x of few bits, zeros among them: later parts are 0
        xs, as_ = rng.integers(-1, 2, (M, K)), rng.integers(-1, 2, (L, r, K))
        as_[:, 3] = 0
    else:
        xs, as_ = rng.standard_normal((M, K)), rng.standard_normal((L, r, K))
        if values == "far":                                      # values 2^-45 of their row's largest
            as_ *= np.where(np.arange(r) % 2, 1.0, 2.0 ** -20)[:, None]
            xs[:, :8] = 0
            as_[:, ::2, 8:] = 0
            xs[:, 0] = 2.0 ** -12
            as_[:, 1::2] *= 2.0 ** 8
    bs = rng.standard_normal((L, N, r))
    odd = rng.random((L, N)) < 0.5                               # rows of B with something infinite
    for l, n in np.argwhere(odd):
        at = rng.choice(r, 1 + (n % 3 == 0), replace=False)
        bs[l, n, at] = rng.choice([np.inf, -np.inf], len(at))
    bs[:, 5, 1], odd[:, 5] = np.nan, True
    x, xe = on_gpu(torch, xs, dtype)
    a, ae = on_gpu(torch, as_, dtype)
    b, be = on_gpu(torch, bs, dtype)
    base, basee = on_gpu(torch, rng.standard_normal((M, N)), dtype)
    ids = rng.integers(-1, L, M)
    scales = np.float32(rng.choice([-1.5, 2.0], L))
    offsets, rows, _ = W.wqbmm_group_rows(torch.from_numpy(ids.astype(np.int32)).cuda(), L)
    y = W.wqbmm_lora_matmul(x, a, b, offsets, rows, scales=torch.from_numpy(scales).cuda(), base=base)
    got = y.double().cpu().numpy()
    want = definition(xe, ae, be, ids, scales.astype(float), basee)
    assert np.isinf(want).any() and np.isnan(want).any() and np.isfinite(want).any()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.where(np.isinf(want), got, 0), np.where(np.isinf(want), want, 0))
    clean, bound = G.lora(xe, ae, finite(be), ids, scales.astype(float), basee, dtype)
    left = np.isfinite(want)                                     # nothing infinite has touched these
    assert np.array_equal(left, ~odd[ids] | (ids < 0)[:, None])
    # fp16 ends at 65504; values from half a step beyond, 65520, round to an infinity
    most = 65520.0 if dtype == "fp16" else np.inf
    close, beyond = np.abs(got - clean) <= bound, got == np.sign(clean) * np.inf
    assert np.where(np.abs(clean) - bound >= most, beyond, close | beyond & (np.abs(clean) + bound >= most))[left].all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [30, 1100])
def test_infinities_in_a_and_x(torch, M, dtype):  # noqa: F811
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(M)
    L, r, K, N = 2, 16, 64, 72
    xs, as_, bs = rng.integers(-2, 3, (M, K)) * 1.0, rng.integers(-2, 3, (L, r, K)) * 1.0, rng.integers(-2, 3, (L, N, r)) * 1.0
    xs[3, 2], xs[4, 2], xs[5, 1], as_[1, 4, 7] = np.inf, -np.inf, np.nan, -np.inf
    bs[0, 8:, 2], bs[0, 9, 3] = 0.0, np.inf
    x, xe = on_gpu(torch, xs, dtype)
    a, ae = on_gpu(torch, as_, dtype)
    b, be = on_gpu(torch, bs, dtype)
    ids = rng.integers(0, L, M)
    ids[:6] = [0, 1, 0, 0, 0, 0]
    offsets, rows, _ = W.wqbmm_group_rows(torch.from_numpy(ids.astype(np.int32)).cuda(), L)
    got = W.wqbmm_lora_matmul(x, a, b, offsets, rows).double().cpu().numpy()
    want = definition(xe, ae, be, ids, np.ones(L), np.zeros((M, N)))
    assert np.isinf(want).any() and np.isnan(want).any()
    # whole numbers that fp16 holds; bf16 rounds by half a step of 2^-8
    assert np.abs(want[np.isfinite(want)]).max() <= 2048
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
    f = ~np.isnan(want)
    assert np.array_equal(got[f & np.isinf(want)], want[f & np.isinf(want)])
    f &= np.isfinite(want)
    assert (np.abs(got[f] - want[f]) <= (0 if dtype == "fp16" else 2.0 ** -8) * np.abs(want[f])).all()
