"""The MXFP4 operators on the GPU against their definitions in 64 bits
(mx_reference.py, which also derives the tolerances)."""
import numpy as np
import pytest

import mx_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    t = pytest.importorskip("torch")
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_msd_amd as W
    W.lib()
    return t


def dt(torch, name):
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[name]


def on_gpu(torch, x, name):
    """x (numpy, 64 bits) rounded to the type, on the GPU, and its exact values."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(torch.float32).to(dt(torch, name))
    return t.cuda(), t.double().numpy()


def bits(torch, t):
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32)


def same(torch, a, b):
    return torch.equal(bits(torch, a), bits(torch, b))


def random_weights(rng, shape, spread=3, zero_blocks=0.05):
    """Codes and scales near those of weights: mostly within a few powers of two, some blocks zero."""
    codes = rng.integers(0, 256, (*shape[:-1], shape[-1] // 2), dtype=np.uint8)
    scales = rng.integers(119 - spread, 120 + spread, (*shape[:-1], shape[-1] // 32)).astype(np.uint8)
    zero = rng.random(scales.shape) < zero_blocks
    codes = np.where(np.repeat(zero, 16, -1), codes & 0x88, codes)      # +0 and -0
    return codes, np.where(zero, rng.integers(0, 255, scales.shape), scales).astype(np.uint8)


def shifted(scales, by):
    """The ordinary blocks' scales moved by a power of two (zero blocks have any)."""
    return np.where((scales > 100) & (scales < 130), scales.astype(int) + by, scales).astype(np.uint8)


def tiled(torch, codes, scales):
    import weight_only_quantized_msd_amd as W
    return W.wqbmm_mxfp4_tile_weights(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())


def check(y, want, bound):
    y = y.double().cpu().numpy()
    assert np.array_equal(np.isnan(y), np.isnan(want))
    ok = np.isnan(want) | (np.abs(y - want) <= bound)
    assert ok.all(), (np.argwhere(~ok)[:4], y[~ok][:4], want[~ok][:4], bound[~ok][:4])


# ---- quantise and read back ------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("M,K,pad", [(1, 32, 0), (1, 4096, 0), (3, 96, 8), (17, 4128, 0), (257, 160, 24), (64, 11008, 8)])
def test_quantize_matches_the_definition(torch, dtype, M, K, pad):
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(M * K + pad)
    x = rng.standard_normal((M, K + pad)) * 2.0 ** rng.integers(-6, 6, (M, 1))
    g, exact = on_gpu(torch, x, dtype)
    g, exact = g[:, :K], exact[:, :K]
    codes, scales = W.wqbmm_mxfp4_quantize(g)
    want_codes, want_scales = R.quantize(exact)
    assert np.array_equal(scales.cpu().numpy(), want_scales)
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    back = torch.full((M, K + pad), 7.0, dtype=g.dtype, device="cuda")
    W.wqbmm_mxfp4_dequantize(codes, scales, g.dtype, y=back[:, :K])
    want = torch.from_numpy(R.dequantize(want_codes, want_scales)).to(torch.float32).to(g.dtype)
    assert same(torch, back[:, :K].cpu().contiguous(), want)
    assert (back[:, K:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_quantize_every_16_bit_value(torch, dtype):
    """Each of the 65536 patterns beside a block maximum of 6 * 2^e for several e, and alone."""
    import weight_only_quantized_msd_amd as W
    pat = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dt(torch, dtype))
    tops = [6.0, 4.0, 7.5, 2.0 ** -8, 0.0] if dtype == "fp16" else [6.0, 4.0, 7.5, 2.0 ** 60, 2.0 ** -120, 0.0]
    for top in tops:
        x = torch.zeros(65536, 32, dtype=pat.dtype)
        x[:, 5], x[:, 20] = pat, top
        codes, scales = W.wqbmm_mxfp4_quantize(x.cuda())
        want_codes, want_scales = R.quantize(x.double().numpy())
        assert np.array_equal(scales.cpu().numpy(), want_scales)
        assert np.array_equal(codes.cpu().numpy(), want_codes)


def test_quantize_fp32_borders(torch):
    """Halfway points and their neighbours, both ends of the range, subnormals, infinities and NaN."""
    import weight_only_quantized_msd_amd as W
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], np.float32)
    vals = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(9))])
    rows = []
    for e in (0, 1, -20, 100, 125, -100, -124, -126, -140):
        row = np.zeros(64, np.float32)
        row[:27] = vals * np.float32(2.0 ** e) if e > -126 else (vals.astype(np.float64) * 2.0 ** e).astype(np.float32)
        row[27] = np.float32(6 * 2.0 ** e)
        rows.append(row)
        rows.append(-row)
    for bad in (np.inf, -np.inf, np.nan):
        row = np.ones(64, np.float32)
        row[40] = bad
        rows.append(row)
    x = np.stack(rows)
    codes, scales = W.wqbmm_mxfp4_quantize(torch.from_numpy(x).cuda())
    want_codes, want_scales = R.quantize(x)
    assert np.array_equal(scales.cpu().numpy(), want_scales)
    assert np.array_equal(codes.cpu().numpy(), want_codes)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_dequantize_all_codes_and_scales(torch, dtype):
    import weight_only_quantized_msd_amd as W
    codes = np.zeros((256, 16), np.uint8)
    codes[:, :8] = np.arange(16).reshape(8, 2) @ [1, 16]
    codes[:, 8:] = codes[:, 7::-1]
    scales = np.arange(256, dtype=np.uint8)[:, None]
    y = W.wqbmm_mxfp4_dequantize(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), dt(torch, dtype))
    want = torch.from_numpy(R.dequantize(codes, scales)).to(torch.float32).to(dt(torch, dtype)).cpu()
    y = y.cpu()
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert same(torch, torch.nan_to_num(y, 0, posinf=float("inf"), neginf=-float("inf")),
                torch.nan_to_num(want, 0, posinf=float("inf"), neginf=-float("inf")))


def test_offsets_past_32_bits(torch):
    """More than 2^32 elements: the last rows are quantised, read back and multiplied as alone."""
    import weight_only_quantized_msd_amd as W
    M, K = 2 ** 17 + 3, 32768
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").fill_(1.5)
    torch.manual_seed(0)
    x[-5:] = torch.randn(5, K, device="cuda").bfloat16()
    codes, scales = W.wqbmm_mxfp4_quantize(x)
    c5, s5 = W.wqbmm_mxfp4_quantize(x[-5:].clone())
    assert torch.equal(codes[-5:], c5) and torch.equal(scales[-5:], s5)
    want_codes, want_scales = R.quantize(x[-5:].double().cpu().numpy())
    assert np.array_equal(c5.cpu().numpy(), want_codes) and np.array_equal(s5.cpu().numpy(), want_scales)
    back = torch.empty_like(x)
    W.wqbmm_mxfp4_dequantize(codes, scales, torch.bfloat16, y=back)
    assert torch.equal(back[-5:], W.wqbmm_mxfp4_dequantize(c5, s5, torch.bfloat16))
    assert (back[:-5:4099] == 1.5).all()
    del back, codes, scales
    rng = np.random.default_rng(1)
    wc, ws = random_weights(rng, (16, K))
    w = tiled(torch, wc, ws)
    for act in ("16bit", "mxfp4"):
        y = W.wqbmm_mxfp4_matmul(x, w, 16, activations=act)
        xe = x[-5:].double().cpu().numpy()
        if act == "mxfp4":
            xe = R.dequantize(*R.quantize(xe))
        check(y[-5:], *R.matmul(xe, R.dequantize(wc, ws), "bf16"))


# ---- products ----------------------------------------------------------------------------

SHAPES = [  # M, K, N, row padding
    (1, 32, 1, 0), (1, 4096, 256, 0), (2, 96, 17, 8), (5, 160, 33, 0), (16, 1056, 100, 0), (17, 544, 63, 8),
    (31, 2080, 48, 0), (33, 512, 130, 0), (64, 640, 34, 24), (65, 32, 16, 0), (65, 4128, 131, 0), (127, 64, 129, 8),
    (128, 1024, 128, 0), (130, 672, 260, 0), (200, 96, 17, 0), (257, 2176, 385, 8), (384, 8192, 64, 0),
]


@pytest.mark.parametrize("act", ["16bit", "mxfp4"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N,pad", SHAPES)
def test_matmul(torch, act, dtype, M, K, N, pad):
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(M * 7 + K * 3 + N)
    g, exact = on_gpu(torch, rng.standard_normal((M, K + pad)), dtype)
    g, exact = g[:, :K], exact[:, :K]
    if pad:
        g = torch.cat([g, torch.full((M, pad), float("nan"), dtype=g.dtype, device="cuda")], 1)[:, :K]
    codes, scales = random_weights(rng, (N, K))
    w = tiled(torch, codes, scales)
    if act == "mxfp4":
        exact = R.dequantize(*R.quantize(exact))
    want, bound = R.matmul(exact, R.dequantize(codes, scales), dtype)
    y = torch.full((M, N), float("nan"), dtype=g.dtype, device="cuda")
    W.wqbmm_mxfp4_matmul(g, w, N, activations=act, y=y)
    check(y, want, bound)
    for _ in range(2):
        assert same(torch, W.wqbmm_mxfp4_matmul(g, w, N, activations=act), y)


@pytest.mark.parametrize("act", ["16bit", "mxfp4"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [3, 40, 150])
def test_matmul_with_scales_beyond_fp16(torch, act, dtype, M):
    """Blocks whose weights no fp16 number holds: far smaller and far larger ones side by side."""
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(M)
    K, N = 608, 150
    codes, scales = random_weights(rng, (N, K))
    scales[0] = rng.integers(60, 104, K // 32)           # whole rows below, above, and across
    scales[40] = rng.integers(141, 170, K // 32)
    scales[70] = rng.integers(100, 145, K // 32)
    x = rng.standard_normal((M, K)) * 2.0 ** -12
    x[0, ::2] = 0
    g, exact = on_gpu(torch, x, dtype)
    if act == "mxfp4":
        exact = R.dequantize(*R.quantize(exact))
    want, bound = R.matmul(exact, R.dequantize(codes, scales), dtype)
    top = 65504.0 if dtype == "fp16" else 3e38
    assert (np.abs(want)[:, 40] > 2 ** 5).any()
    fits = np.abs(want) + bound < top
    y = W.wqbmm_mxfp4_matmul(g, tiled(torch, codes, scales), N, activations=act).double().cpu().numpy()
    assert (np.abs(y - want) <= bound)[fits].all()
    assert np.isinf(y[np.abs(want) - bound > 1.01 * top]).all()


@pytest.mark.parametrize("act", ["16bit", "mxfp4"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [4, 70])
def test_matmul_nan_and_infinity_stay_in_their_rows_and_columns(torch, act, dtype, M):
    import weight_only_quantized_msd_amd as W
    rng = np.random.default_rng(9)
    K, N = 288, 50
    codes, scales = random_weights(rng, (N, K), zero_blocks=0)
    codes |= 0x11                                        # no zero weights: infinity times any is infinity
    scales[7, 3] = 255                                   # column 7 is NaN
    x = rng.standard_normal((M, K))
    x[1, 280], x[2, 5] = np.nan, np.inf
    g, exact = on_gpu(torch, x, dtype)
    for wide in (False, True):
        if wide:
            scales[20, 0] = 90                           # not exact in fp16
        y = W.wqbmm_mxfp4_matmul(g, tiled(torch, codes, scales), N, activations=act).double().cpu().numpy()
        assert np.isnan(y[1]).all() and np.isnan(y[:, 7]).all()
        others = np.arange(N) != 7
        if act == "16bit":
            w = R.dequantize(codes, scales)
            assert np.array_equal(y[2][others], np.sign(w[others, 5]) * np.inf)
        else:
            assert np.isnan(y[2]).all()
        rest = np.setdiff1d(np.arange(M), [1, 2])
        e = exact[rest] if act == "16bit" else R.dequantize(*R.quantize(exact[rest]))
        want, bound = R.matmul(e, R.dequantize(codes, scales)[others], dtype)
        assert (np.abs(y[rest][:, others] - want) <= bound).all()


@pytest.mark.parametrize("act", ["16bit", "mxfp4"])
@pytest.mark.parametrize("M", [1, 64, 100])
def test_matmul_zero_rows_give_zero(torch, act, M):
    import weight_only_quantized_msd_amd as W
    codes, scales = random_weights(np.random.default_rng(2), (40, 256))
    w = tiled(torch, codes, scales)
    y = W.wqbmm_mxfp4_matmul(torch.zeros(M, 256, dtype=torch.float16, device="cuda"), w, 40, activations=act)
    assert (y == 0).all()
    assert W.wqbmm_mxfp4_matmul(torch.zeros(0, 256, dtype=torch.float16, device="cuda"), w, 40,
                                activations=act).shape == (0, 40)


def test_stacked_weights_are_tiled_one_after_another(torch):
    import weight_only_quantized_msd_amd as W
    codes, scales = random_weights(np.random.default_rng(3), (3, 32, 160))
    whole = tiled(torch, codes, scales)
    flat = tiled(torch, codes.reshape(96, 80), scales.reshape(96, 5))
    assert torch.equal(whole, flat)
    with pytest.raises(ValueError, match="N % 16"):
        tiled(torch, codes[:, :17].copy(), scales[:, :17].copy())


# ---- mixture of experts --------------------------------------------------------------------

def moe_case(torch, T, H, inter, E, k, dtype, seed, scale_shift=0):
    rng = np.random.default_rng(seed)
    gu = random_weights(rng, (E, 2 * inter, H))
    dn = random_weights(rng, (E, H, inter))
    gu = (gu[0], shifted(gu[1], scale_shift))
    # normal logits of the size that separates them well beyond fp32's error
    for attempt in range(50):
        x, xe = on_gpu(torch, rng.standard_normal((T, H)), dtype)
        router, re = on_gpu(torch, rng.standard_normal((E, H)) * 2 * H ** -0.5, dtype)
        _, _, gap, slack = R.route(xe, re, k, True)
        if gap > 4 * slack:
            return x, xe, router, re, gu, dn
    raise AssertionError("no inputs whose experts are clear")


MOE_SHAPES = [  # T, H, I, E, k
    (1, 32, 32, 1, 1), (1, 512, 256, 64, 8), (2, 160, 96, 5, 5), (3, 1056, 64, 8, 2), (16, 256, 736, 12, 3),
    (17, 128, 160, 4, 1), (33, 288, 96, 6, 2), (64, 128, 64, 3, 2), (64, 64, 32, 256, 4), (7, 4096, 544, 9, 2),
    (40, 96, 2208, 20, 16),
]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,H,inter,E,k", MOE_SHAPES)
def test_moe(torch, renorm, dtype, T, H, inter, E, k):
    import weight_only_quantized_msd_amd as W
    x, xe, router, re, gu, dn = moe_case(torch, T, H, inter, E, k, dtype, T + H + inter)
    want, bound, ids, weights, wbound, _, _ = R.moe(xe, re, R.dequantize(*gu), R.dequantize(*dn), k, renorm, dtype)
    gt, dt_ = tiled(torch, *gu), tiled(torch, *dn)
    y, got_ids, got_weights = W.wqbmm_mxfp4_moe(x, router, gt, dt_, inter, k, renormalize=renorm)
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    assert (np.abs(got_weights.double().cpu().numpy() - weights) <= wbound).all()
    check(y, want, bound)
    y2, ids2, weights2 = W.wqbmm_mxfp4_moe(x, router, gt, dt_, inter, k, renormalize=renorm)
    assert same(torch, y, y2) and torch.equal(ids2, got_ids) and same(torch, weights2, got_weights)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_moe_weights_beyond_fp16(torch, dtype):
    import weight_only_quantized_msd_amd as W
    T, H, inter, E, k = 20, 160, 64, 4, 2
    x, xe, router, re, gu, dn = moe_case(torch, T, H, inter, E, k, dtype, 5)
    gu[1][:, :inter] = shifted(gu[1][:, :inter], -20)    # tiny gates, ordinary up rows
    want, bound, *_ = R.moe(xe, re, R.dequantize(*gu), R.dequantize(*dn), k, True, dtype)
    y, _, _ = W.wqbmm_mxfp4_moe(x, router, tiled(torch, *gu), tiled(torch, *dn), inter, k)
    check(y, want, bound)


def test_moe_large_intermediate_values(torch):
    """fp16 tokens whose products of gate and up are beyond fp16, the output within it."""
    import weight_only_quantized_msd_amd as W
    T, H, inter, E, k = 3, 128, 64, 2, 1
    x, xe, router, re, gu, dn = moe_case(torch, T, H, inter, E, k, "fp16", 6, scale_shift=14)
    dn = (dn[0], shifted(dn[1], -18))
    want, bound, *_ = R.moe(xe, re, R.dequantize(*gu), R.dequantize(*dn), k, True, "fp16")
    g = R.dequantize(*gu)[0] @ xe[0]
    assert np.abs(g).max() ** 2 > 65504 and np.abs(want).max() < 65504
    y, _, _ = W.wqbmm_mxfp4_moe(x, router, tiled(torch, *gu), tiled(torch, *dn), inter, k)
    check(y, want, bound)


def test_moe_ties_go_to_the_lowest_expert_and_nan_stays_in_its_token(torch):
    import weight_only_quantized_msd_amd as W
    T, H, inter, E, k = 5, 64, 32, 70, 3
    x, xe, router, re, gu, dn = moe_case(torch, T, H, inter, E, k, "fp16", 7)
    router[:] = router[:1]                               # all logits equal
    y, ids, weights = W.wqbmm_mxfp4_moe(x, router, tiled(torch, *gu), tiled(torch, *dn), inter, k)
    assert (ids.cpu() == torch.arange(k, dtype=torch.int32)).all()
    assert (weights.cpu() - 1 / 3).abs().max() <= 2 * 2.0 ** -24
    clean = y.clone()
    x[2, 9] = float("nan")
    y, ids, weights = W.wqbmm_mxfp4_moe(x, router, tiled(torch, *gu), tiled(torch, *dn), inter, k)
    assert torch.isnan(y[2]).all() and torch.isnan(weights[2]).all()
    assert ((ids >= 0) & (ids < E)).all()
    keep = [0, 1, 3, 4]
    assert same(torch, y[keep], clean[keep])


def test_moe_strided_rows_and_empty_batch(torch):
    import weight_only_quantized_msd_amd as W
    T, H, inter, E, k = 6, 96, 64, 4, 2
    x, xe, router, re, gu, dn = moe_case(torch, T, H, inter, E, k, "bf16", 8)
    gt, dn_t = tiled(torch, *gu), tiled(torch, *dn)
    wide = torch.full((T, H + 40), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, :H] = x
    a, b = W.wqbmm_mxfp4_moe(x, router, gt, dn_t, inter, k), W.wqbmm_mxfp4_moe(wide[:, :H], router, gt, dn_t, inter, k)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    y, ids, weights = W.wqbmm_mxfp4_moe(x[:0], router, gt, dn_t, inter, k)
    assert y.shape == (0, H) and ids.shape == (0, k)


# ---- streams, graphs, refusals -----------------------------------------------------------------

def block(W, x, w, N, router, gt, dn, inter, k):
    """Every operator once, with workspace of several sizes."""
    codes, scales = W.wqbmm_mxfp4_quantize(x)
    back = W.wqbmm_mxfp4_dequantize(codes, scales, x.dtype)
    outs = [codes, scales, back]
    for act in ("16bit", "mxfp4"):
        outs += [W.wqbmm_mxfp4_matmul(x[:9], w, N, activations=act), W.wqbmm_mxfp4_matmul(x, w, N, activations=act)]
    outs += W.wqbmm_mxfp4_moe(x[:5], router, gt, dn, inter, k)
    return outs


@pytest.fixture(scope="module")
def block_inputs(torch):
    T, H, inter, E, k, N = 100, 640, 96, 6, 2, 72
    x, _, router, _, gu, dn = moe_case(torch, T, H, inter, E, k, "fp16", 11)
    w = tiled(torch, *random_weights(np.random.default_rng(4), (N, H)))
    return x, w, N, router, tiled(torch, *gu), tiled(torch, *dn), inter, k


def test_another_stream(torch, block_inputs):
    import weight_only_quantized_msd_amd as W
    want = block(W, *block_inputs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = block(W, *block_inputs)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # as an argument: outputs belong to that stream
    x, w, N = block_inputs[:3]
    y = W.wqbmm_mxfp4_matmul(x, w, N, activations="mxfp4", stream=side)
    side.synchronize()
    assert torch.equal(y, want[6])


def test_graph_replays(torch, block_inputs):
    import weight_only_quantized_msd_amd as W
    x, *rest = block_inputs
    x = x.clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        block(W, x, *rest)                               # workspace grows before the capture
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = block(W, x, *rest)
    torch.cuda.synchronize()
    torch.manual_seed(5)
    for i in range(4):
        x.copy_(torch.randn_like(x))
        torch.cuda.synchronize()
        want = block(W, x, *rest)                        # the default stream's workspace
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs)), i


def test_growth_during_capture_is_refused(torch, block_inputs):
    import weight_only_quantized_msd_amd as W
    x, w, N = block_inputs[:3]
    s = torch.cuda.Stream()
    y = torch.full((x.shape[0], N), 3.0, dtype=x.dtype, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin()
        try:
            y.mul_(1.0)
            with pytest.raises(W.WqbmmError) as e:
                W.wqbmm_mxfp4_matmul(x, w, N, activations="mxfp4", y=y)
        finally:
            graph.capture_end()
    torch.cuda.synchronize()
    assert e.value.status == W.WQBMM_ERR_CAPTURE and (y == 3.0).all()


def test_prepared_operands_of_the_int4_path_are_not_mistaken(torch, block_inputs):
    """Its stage 2 refuses to run on operands that one of these calls has overwritten."""
    import weight_only_quantized_msd_amd as W
    from weight_only_quantized_msd_amd import datagen
    d = datagen.random_case(256, 512, 256, 128, seed=1)
    x, s = torch.from_numpy(d["x"]).cuda(), torch.from_numpy(d["scale"]).cuda()
    w = W.wqbmm_a16w4_tile_weights(torch.from_numpy(d["w_packed"]).cuda())
    ref = W.wqbmm_a16w4_msd(x, w, s, 128)
    assert same(torch, W.wqbmm_a16w4_msd_profile_stage(x, w, s, 128, 2), ref)
    W.wqbmm_mxfp4_matmul(block_inputs[0], block_inputs[1], block_inputs[2], activations="mxfp4")
    with pytest.raises(W.WqbmmError):
        W.wqbmm_a16w4_msd_profile_stage(x, w, s, 128, 2)
    assert same(torch, W.wqbmm_a16w4_msd(x, w, s, 128), ref)


def test_wrapper_refusals(torch, block_inputs):
    import weight_only_quantized_msd_amd as W
    x, w, N, router, gt, dn, inter, k = block_inputs
    codes, scales = W.wqbmm_mxfp4_quantize(x)
    bad = [
        (ValueError, lambda: W.wqbmm_mxfp4_quantize(x.t())),
        (ValueError, lambda: W.wqbmm_mxfp4_quantize(x[0])),
        (TypeError, lambda: W.wqbmm_mxfp4_quantize(x.double())),
        (W.WqbmmError, lambda: W.wqbmm_mxfp4_quantize(x[:, :40])),              # K % 32
        (W.WqbmmError, lambda: W.wqbmm_mxfp4_quantize(x[:, 1:33])),             # misaligned
        (W.WqbmmError, lambda: W.wqbmm_mxfp4_quantize(torch.zeros(4, 36, device="cuda")[:, :32])),   # rows 36 apart
        (ValueError, lambda: W.wqbmm_mxfp4_quantize(x, codes=codes[:, :-1])),
        (ValueError, lambda: W.wqbmm_mxfp4_dequantize(codes, scales[:, :-1], x.dtype)),
        (TypeError, lambda: W.wqbmm_mxfp4_dequantize(codes, scales, torch.int8)),
        (ValueError, lambda: W.wqbmm_mxfp4_dequantize(codes, scales, x.dtype, y=x[:-1])),
        (ValueError, lambda: W.wqbmm_mxfp4_tile_weights(codes, scales[:-1])),
        (ValueError, lambda: W.wqbmm_mxfp4_matmul(x, w, N + 16)),
        (ValueError, lambda: W.wqbmm_mxfp4_matmul(x, w, N, activations="fp8")),
        (TypeError, lambda: W.wqbmm_mxfp4_matmul(x.float(), w, N)),
        (ValueError, lambda: W.wqbmm_mxfp4_matmul(x, w, N, y=torch.empty_like(x))),
        (W.WqbmmError, lambda: W.wqbmm_mxfp4_matmul(x, w, 0)),
        (ValueError, lambda: W.wqbmm_mxfp4_moe(x[:5], router[:, :-32], gt, dn, inter, k)),
        (ValueError, lambda: W.wqbmm_mxfp4_moe(x[:5], router.bfloat16(), gt, dn, inter, k)),
        (ValueError, lambda: W.wqbmm_mxfp4_moe(x[:5], router, dn, gt, inter, k)),
        (W.WqbmmError, lambda: W.wqbmm_mxfp4_moe(x[:65], router, gt, dn, inter, k)),
        (W.WqbmmError, lambda: W.wqbmm_mxfp4_moe(x[:5], router, gt, dn, inter, 0)),
        (W.WqbmmError, lambda: W.wqbmm_mxfp4_moe(x[:5], router, gt, dn, inter, 7)),
    ]
    for i, (kind, f) in enumerate(bad):
        with pytest.raises(kind):
            f()
            raise AssertionError(f"call {i} was let through")
