"""The operators whose weights depend on the row on the GPU: results beyond the 2^32
threads of a launch."""
import pytest

from test_gpu_mxfp4 import bits, random_weights, tiled, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room(torch):  # noqa: F811
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 * 2 ** 30:
        pytest.skip("needs 100 GB")
    yield
    torch.cuda.empty_cache()


def test_combine_beyond_a_launch(torch):  # noqa: F811
    """y of 64 GB: k = 1, so that a value is one product, rounded to fp32 and then to 16 bits as torch does it."""
    import weight_only_quantized_msd_amd as W
    T, H, S = 2 ** 22 + 3, 2 ** 13, 1000
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn(S, H, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.randint(0, S, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    weights = torch.rand(T, 1, generator=g, device="cuda")
    y = W.wqbmm_moe_combine(z, slots, weights)
    for t in range(0, T, 2 ** 17):
        some = slice(t, min(T, t + 2 ** 17))
        want = (z[slots[some, 0].long()].float() * weights[some]).to(torch.bfloat16)
        assert torch.equal(y[some], want), t


def test_grouped_product_beyond_a_launch(torch):  # noqa: F811
    """2^24 places of three far rows: each holds one of the fifteen results that a small call gives."""
    import numpy as np
    import weight_only_quantized_msd_amd as W
    S, R, groups, K, N, ld = 2 ** 24, 3, 5, 32, 2 ** 11, 2 ** 29
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty((R - 1) * ld + K, dtype=torch.bfloat16, device="cuda").as_strided((R, K), (ld, 1))
    x.copy_(torch.randn(R, K, generator=g, device="cuda"))
    w = tiled(torch, *random_weights(np.random.default_rng(3), (groups, N, K)))
    each = torch.arange(groups * R, device="cuda", dtype=torch.int32)
    table = W.wqbmm_mxfp4_grouped_matmul(x, w, R * torch.arange(groups + 1, device="cuda", dtype=torch.int32), N,
                                         rows=each % R, gated=True)
    ids = torch.randint(0, groups, (S,), generator=g, device="cuda", dtype=torch.int32)
    offsets, _, _ = W.wqbmm_group_rows(ids, groups)
    rows = torch.randint(0, R, (S,), generator=g, device="cuda", dtype=torch.int32)
    y = W.wqbmm_mxfp4_grouped_matmul(x, w, offsets, N, rows=rows, gated=True)
    place = torch.arange(S, device="cuda")
    at = (torch.searchsorted(offsets.long(), place, right=True) - 1) * R + rows
    for s in range(0, S, 2 ** 20):
        some = slice(s, s + 2 ** 20)
        assert torch.equal(bits(torch, y[some]), bits(torch, table[at[some]])), s
