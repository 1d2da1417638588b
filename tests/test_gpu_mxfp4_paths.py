"""The MXFP4 operators at the sizes where another kernel, tile or way of reading
takes over, against their definitions in 64 bits (mx_reference.py, which also
derives the tolerances).  Large products are compared on some of their rows."""
import numpy as np
import pytest

import mx_reference as R
from test_gpu_mxfp4 import check, dt, moe_case, on_gpu, random_weights, same, tiled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_msd_amd as W
    W.lib()
    return t


def some_rows(rng, M):
    """The first and last rows, those beside a multiple of 64, and others."""
    edges = [m for b in range(64, M, 64) for m in (b - 1, b)]
    return np.unique(np.concatenate([[0, M - 1], rng.choice(edges, min(8, len(edges)), replace=False),
                                     rng.integers(0, M, 16)]).astype(int))


# Tiled products: every tile, with and without K-splits; K ends inside a K-tile,
# inside a quad of them and after a number of K-tiles of every remainder by 3 and 4;
# N odd, even, a multiple of 4 and of 8; M inside a tile.
TILED = [
    (65, 32, 17), (65, 1056, 17), (100, 2080, 40), (130, 160, 33), (193, 416, 132), (129, 928, 72), (300, 4128, 36),
    (777, 288, 1000), (1000, 544, 516), (90, 8224, 64), (1500, 2080, 4099), (1500, 2208, 4104), (1030, 3680, 4100),
    (1100, 2912, 3970), (2500, 1056, 6000), (2500, 2080, 4099), (2300, 1952, 4136),
]


@pytest.mark.parametrize("act", ["16bit", "mxfp4"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N", TILED)
def test_tiled_products(torch, act, dtype, M, K, N):
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(M + K + N)
    x, exact = on_gpu(torch, rng.standard_normal((M, K)), dtype)
    # rows wider than they are long: what stands beside them is never used
    wide = torch.full((M, K + 24), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, :K] = x
    codes, scales = random_weights(rng, (N, K))
    w = tiled(torch, codes, scales)
    rows = some_rows(rng, M)
    e = exact[rows]
    if act == "mxfp4":
        e = R.dequantize(*R.quantize(e))
    y = torch.full((M, N), float("nan"), dtype=x.dtype, device="cuda")
    W.wqbmm_mxfp4_matmul(wide[:, :K], w, N, activations=act, y=y)
    assert not torch.isnan(y).any()
    check(y[torch.from_numpy(rows).cuda()], *R.matmul(e, R.dequantize(codes, scales), dtype))
    # the same rows in another order and the same columns come out the same
    again = W.wqbmm_mxfp4_matmul(x.flip(0), w, N, activations=act)
    assert same(torch, again.flip(0), y)


@pytest.mark.parametrize("M,K,N", [(1500, 2080, 4099), (1030, 3680, 4100), (700, 544, 1000)])
def test_tiled_products_with_scales_beyond_fp16(torch, M, K, N):
    """fp16 rows whose tile holds some weights that no fp16 number does."""
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(M)
    codes, scales = random_weights(rng, (N, K))
    scales[N // 2] = rng.integers(95, 104, K // 32)
    x, exact = on_gpu(torch, rng.standard_normal((M, K)), "fp16")
    rows = some_rows(rng, M)
    y = W.wqbmm_mxfp4_matmul(x, tiled(torch, codes, scales), N)
    check(y[torch.from_numpy(rows).cuda()], *R.matmul(exact[rows], R.dequantize(codes, scales), "fp16"))


# Few rows: one, two and four tiles of 16 rows; one to four panels a workgroup.
FEW = [(1, 4096, 4112), (7, 1056, 8200), (16, 544, 12300), (17, 2080, 4112), (32, 160, 12300), (33, 544, 8200),
       (48, 1184, 12300), (64, 96, 16400), (50, 6176, 4112), (64, 4128, 130)]


@pytest.mark.parametrize("act", ["16bit", "mxfp4"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N", FEW)
def test_few_rows(torch, act, dtype, M, K, N):
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(M + K + N)
    x, exact = on_gpu(torch, rng.standard_normal((M, K)), dtype)
    codes, scales = random_weights(rng, (N, K))
    if act == "mxfp4":
        exact = R.dequantize(*R.quantize(exact))
    y = W.wqbmm_mxfp4_matmul(x, tiled(torch, codes, scales), N, activations=act)
    check(y, *R.matmul(exact, R.dequantize(codes, scales), dtype))


@pytest.mark.parametrize("act", ["16bit", "mxfp4"])
def test_rows_far_apart(torch, act):
    """Rows of x 2^22 values apart, more than the tiled product addresses."""
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(3)
    M, K, N = 131, 288, 72
    x, _ = on_gpu(torch, rng.standard_normal((M, K)), "bf16")
    far = torch.empty(M, 2 ** 22, dtype=x.dtype, device="cuda")
    far[:, :K] = x
    codes, scales = random_weights(rng, (N, K))
    w = tiled(torch, codes, scales)
    e = x.double().cpu().numpy()
    if act == "mxfp4":
        e = R.dequantize(*R.quantize(e))
    check(W.wqbmm_mxfp4_matmul(far[:, :K], w, N, activations=act), *R.matmul(e, R.dequantize(codes, scales), "bf16"))


# ---- mixture of experts ------------------------------------------------------------------

def clear_case(torch, T, H, inter, E, k, dtype, seed):
    """As moe_case, with logits that are 1/8 apart: expert e's is x[t][e]."""
    if E > H:
        return moe_case(torch, T, H, inter, E, k, dtype, seed)
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H))
    x[:, :E] = rng.permuted(np.tile(np.arange(E) / 8 - E / 16, (T, 1)), axis=1)
    x, xe = on_gpu(torch, x, dtype)
    router, re = on_gpu(torch, np.eye(E, H), dtype)
    _, _, gap, slack = R.route(xe, re, k, True)
    assert E == 1 or gap > 4 * slack
    return x, xe, router, re, random_weights(rng, (E, 2 * inter, H)), random_weights(rng, (E, H, inter))


MOE = [  # T, H, I, E, k: tokens by themselves and together; all rows with the same experts; staged and direct rows; slots by pair and by expert
    (1, 96, 64, 256, 16), (1, 2080, 1056, 3, 3), (1, 512, 2592, 70, 1), (64, 96, 2080, 2, 2), (64, 160, 96, 1, 1),
    (50, 64, 2208, 3, 1), (20, 2048, 64, 40, 4), (64, 2080, 32, 33, 2), (2, 4096, 32, 200, 16), (5, 1056, 4128, 6, 2),
    (33, 544, 1056, 4, 3), (64, 224, 96, 5, 2), (64, 320, 64, 2, 1), (40, 416, 32, 16, 3), (17, 736, 96, 256, 8),
    (16, 1056, 96, 90, 4), (16, 768, 96, 90, 6), (9, 1184, 2080, 12, 1), (24, 512, 224, 4, 1),
]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,H,inter,E,k", MOE)
def test_moe_paths(torch, renorm, dtype, T, H, inter, E, k):
    import weight_only_quantized_msd_amd as W
    x, xe, router, re, gu, dn = clear_case(torch, T, H, inter, E, k, dtype, T + H + inter)
    want, bound, ids, weights, wbound, _, _ = R.moe(xe, re, R.dequantize(*gu), R.dequantize(*dn), k, renorm, dtype)
    gt, dn_t = tiled(torch, *gu), tiled(torch, *dn)
    y, got_ids, got_weights = W.wqbmm_mxfp4_moe(x, router, gt, dn_t, inter, k, renormalize=renorm)
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    assert (np.abs(got_weights.double().cpu().numpy() - weights) <= wbound).all()
    check(y, want, bound)
    again = W.wqbmm_mxfp4_moe(x, router, gt, dn_t, inter, k, renormalize=renorm)
    assert same(torch, y, again[0]) and torch.equal(got_ids, again[1]) and same(torch, got_weights, again[2])


@pytest.mark.parametrize("T,H,inter,E,k", [(40, 64, 96, 6, 2), (40, 64, 2080, 6, 2), (1, 64, 96, 6, 2), (40, 384, 96, 6, 2), (40, 384, 2080, 6, 2)])
def test_moe_a_nan_weight_stays_with_its_expert(torch, T, H, inter, E, k):
    import weight_only_quantized_msd_amd as W
    x, xe, router, re, gu, dn = clear_case(torch, T, H, inter, E, k, "bf16", 21)
    clean, ids, _ = W.wqbmm_mxfp4_moe(x, router, tiled(torch, *gu), tiled(torch, *dn), inter, k)
    bad = int(ids[0, 0])
    for which in (gu, dn):
        scales = which[1].copy()
        scales[bad, 3, 0] = 255                              # a gate row: all of y; a row of down: column 3
        weights = [tiled(torch, *gu), tiled(torch, *dn)]
        weights[0 if which is gu else 1] = tiled(torch, which[0], scales)
        y, ids2, _ = W.wqbmm_mxfp4_moe(x, router, *weights, inter, k)
        assert torch.equal(ids, ids2)
        hit = (ids == bad).any(1)
        assert hit.any() and same(torch, y[~hit], clean[~hit])
        assert torch.isnan(y[hit]).all() if which is gu else torch.isnan(y[hit][:, 3]).all()
        if which is dn:
            rest = [c for c in range(H) if c != 3]
            assert same(torch, y[hit][:, rest].contiguous(), clean[hit][:, rest].contiguous())


@pytest.mark.parametrize("values", ["few", "special", "equal"])
@pytest.mark.parametrize("E,k", [(1, 1), (7, 7), (32, 16), (33, 5), (64, 16), (65, 1), (65, 16), (128, 8), (200, 16), (256, 16)])
@pytest.mark.parametrize("T", [1, 2, 64])
def test_moe_choices(torch, T, E, k, values):
    """Larger logits first, NaN above all, -0 equal to +0, equal logits by index; the logits are exact."""
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(E + k)
    H, inter = 64 if T < 64 else 224, 32        # 64 tokens of 224: together
    of = {"few": [-1.0, -0.0, 0.0, 0.5, 3.0], "special": [-np.inf, -2.0, -0.0, 0.0, 1.0, np.inf, np.nan], "equal": [-1.5]}
    logits = rng.choice(of[values], E)
    x, router = np.zeros((T, H)), np.zeros((E, H))
    x[:, 0], router[:, 0] = 1.0, logits
    x, router = on_gpu(torch, x, "bf16")[0], on_gpu(torch, router, "bf16")[0]
    gt, dn = tiled(torch, *random_weights(rng, (E, 2 * inter, H))), tiled(torch, *random_weights(rng, (E, H, inter)))
    key = np.where(np.isnan(logits), np.inf, np.clip(logits, -1e9, 1e9))
    order = np.argsort(-key, kind="stable")[:k]
    for renorm in (True, False):
        _, ids, weights = W.wqbmm_mxfp4_moe(x, router, gt, dn, inter, k, renormalize=renorm)
        assert np.array_equal(ids.cpu().numpy(), np.tile(order, (T, 1)))
        if np.isfinite(logits).all():
            p = np.exp(logits - logits.max())
            p = p[order] / (p[order].sum() if renorm else p.sum())
            # exp and its argument, the division, a sum of E terms: fp32 steps
            assert (np.abs(weights.double().cpu().numpy() - p) <= (E + 16) * 2.0 ** -24 * p).all()


def test_moe_one_token_ties_and_nan(torch):
    import weight_only_quantized_msd_amd as W
    T, H, inter, E, k = 1, 64, 32, 90, 4
    x, xe, router, re, gu, dn = moe_case(torch, T, H, inter, E, k, "bf16", 13)
    gt, dn_t = tiled(torch, *gu), tiled(torch, *dn)
    router[:] = router[:1]
    y, ids, weights = W.wqbmm_mxfp4_moe(x, router, gt, dn_t, inter, k)
    assert ids.tolist() == [[0, 1, 2, 3]] and (weights.cpu() - 0.25).abs().max() <= 2 * 2.0 ** -24
    router[70, 5] = float("nan")                             # a NaN counts as the largest
    y, ids, weights = W.wqbmm_mxfp4_moe(x, router, gt, dn_t, inter, k)
    assert ids.tolist() == [[70, 0, 1, 2]] and torch.isnan(weights).all() and torch.isnan(y).all()


# ---- the two ways into the library -------------------------------------------------------------

def test_given_outputs_and_streams_agree_with_the_ordinary_call(torch):
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(17)
    T, H, inter, E, k, N = 3, 288, 96, 6, 2, 72
    x, _, router, _, gu, dn = clear_case(torch, T, H, inter, E, k, "fp16", 17)
    gt, dn_t = tiled(torch, *gu), tiled(torch, *dn)
    w = tiled(torch, *random_weights(rng, (N, H)))
    current = torch.cuda.current_stream()
    codes, scales = W.wqbmm_mxfp4_quantize(x)
    for a, b in zip((codes, scales), W.wqbmm_mxfp4_quantize(x, stream=current)):
        assert torch.equal(a, b)
    for t in (torch.float16, torch.bfloat16, torch.float32):
        y = W.wqbmm_mxfp4_dequantize(codes, scales, t)
        assert y.dtype == t and torch.equal(y, W.wqbmm_mxfp4_dequantize(codes, scales, t, y=torch.empty_like(y)))
    for act in ("16bit", "mxfp4"):
        assert same(torch, W.wqbmm_mxfp4_matmul(x, w, N, activations=act),
                    W.wqbmm_mxfp4_matmul(x, w, N, activations=act, stream=current))
    for n in (1, 3):
        a = W.wqbmm_mxfp4_moe(x[:n], router, gt, dn_t, inter, k)
        b = W.wqbmm_mxfp4_moe(x[:n], router, gt, dn_t, inter, k, y=torch.empty_like(x[:n]))
        assert same(torch, a[0], b[0]) and torch.equal(a[1], b[1]) and same(torch, a[2], b[2])
    # an argument in the wrong place or of the wrong kind is refused the same way with and without outputs
    for f in (lambda **o: W.wqbmm_mxfp4_matmul(x, w[:-16], N, **o), lambda **o: W.wqbmm_mxfp4_matmul(x, w.cpu(), N, **o),
              lambda **o: W.wqbmm_mxfp4_matmul(x.cpu(), w, N, **o), lambda **o: W.wqbmm_mxfp4_matmul(x[:, ::2], w, N, **o)):
        for o in ({}, {"stream": current}):
            with pytest.raises(ValueError):
                f(**o)


def test_graph_replays_of_the_other_paths(torch):
    """One token, many rows with K-splits, and the tiles without: captured, replayed
    between eager calls, and compared each time."""
    import weight_only_quantized_msd_amd as W
    T, H, inter, E, k, N = 64, 2080, 96, 6, 2, 136
    x, _, router, _, gu, dn = clear_case(torch, T, H, inter, E, k, "bf16", 31)
    gt, dn_t = tiled(torch, *gu), tiled(torch, *dn)
    w = tiled(torch, *random_weights(np.random.default_rng(2), (N, H)))
    big = torch.empty(300, H, dtype=x.dtype, device="cuda")

    def calls():
        outs = []
        for act in ("16bit", "mxfp4"):
            outs += [W.wqbmm_mxfp4_matmul(big[:m], w, N, activations=act) for m in (1, 40, 90, 300)]
        for n in (1, 2, 64):
            outs += W.wqbmm_mxfp4_moe(big[:n], router, gt, dn_t, inter, k)
        return outs

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        big.normal_()
        calls()                                              # workspace grows before the capture
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = calls()
    torch.cuda.synchronize()
    for i in range(4):
        big.normal_()
        torch.cuda.synchronize()
        want = calls()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs)), i


def test_example(torch, capsys):
    """The example's block: the kernels add a rounding, quantising what MXFP4 costs."""
    import importlib.util
    import os
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_block.py")
    spec = importlib.util.spec_from_file_location("mxfp4_block", at)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    report, y, ids, weights = module.main(["--hidden", "256", "--ffn", "352", "--prompt", "70"])
    for name, (cost, added) in report.items():
        # a uniform rounding of at most 2^-8 of the value; each factor in MXFP4 is off by at most a quarter of its value
        assert added <= 2.0 ** -8 and cost <= 0.25 * (2 + 0.25), name
    assert torch.isfinite(y).all() and (weights.sum(1) - 1).abs().max() <= 16 * 2.0 ** -24
    assert "decoding step" in capsys.readouterr().out
