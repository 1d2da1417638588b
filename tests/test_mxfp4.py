"""MXFP4 operators without a GPU: the tests' reference against brute force, and
the refusals of the C ABI and of the wrappers."""
import numpy as np
import pytest

import mx_reference as R
from weight_only_quantized_msd_amd import _lib as L

FAKE = 0x1000          # 16-byte aligned, never dereferenced: validation fails first
MIS = 0x1008           # misaligned
I64_MAX = 2 ** 63 - 1


# ---- the reference ---------------------------------------------------------------

def test_reference_rounds_half_to_even():
    grid = np.arange(0, 8, 1 / 64)
    code = R.nearest_code(grid)
    assert (np.abs(R.MAGNITUDES[code] - np.minimum(grid, 6)) <= np.abs(
        R.MAGNITUDES[None] - np.minimum(grid, 6)[:, None]).min(1)).all()
    for value, want in [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (7.0, 7)]:
        assert R.nearest_code(value) == want


def test_reference_scales_and_packing():
    x = np.zeros((1, 64))
    x[0, 0], x[0, 1], x[0, 33] = 6.0, -3.0, 2.0 ** -140
    codes, scales = R.quantize(x)
    assert scales.tolist() == [[127, 0]]               # 6 = 1.5 * 2^2; the smallest scale
    assert codes[0, 0] == 7 | (13 << 4) and not codes[0, 1:].any()
    assert np.array_equal(R.dequantize(codes, scales)[0, :2], [6.0, -3.0])
    x[0, 40] = np.inf
    codes, scales = R.quantize(x)
    assert scales[0, 1] == 255 and np.isnan(R.dequantize(codes, scales)[0, 32:]).all()


def test_reference_error_is_within_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((8, 256)) * 2.0 ** rng.integers(-30, 30, (8, 1))
    codes, scales = R.quantize(x)
    s = 2.0 ** (np.repeat(scales, 32, -1).astype(float) - 127)
    a = np.abs(x) / s
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, np.where(a <= 6, 1.0, 2.0)))
    assert (np.abs(R.dequantize(codes, scales) - x) <= half * s).all()


# ---- refusals of the C ABI ------------------------------------------------------------

@pytest.fixture
def no_device_visible():
    """As for the other fake-pointer checks: without a GPU a call that
    validation wrongly lets through stops at the device check."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("fake-pointer validation checks run only without a visible GPU")


def call(name, args, over):
    assert set(over) <= set(args), "a test of an argument that is not there"
    return getattr(L.lib(), name)(*[(over.get(k, v) or None) if k in POINTERS else over.get(k, v)
                                    for k, v in args.items()])


POINTERS = {"x", "codes", "scales", "y", "w", "router", "gate_up", "down", "ids", "weights", "stream"}
OK_FOR_A_GPU = L.WQBMM_ERR_UNSUPPORTED                 # arguments are fine, but there is no device

QUANTIZE = dict(x=FAKE, dtype=0, M=3, K=64, ld=64, codes=FAKE, scales=FAKE, stream=0)
DEQUANTIZE = dict(codes=FAKE, scales=FAKE, M=3, K=64, y=FAKE, dtype=0, ld=64, stream=0)
TILE = dict(codes=FAKE, scales=FAKE, K=64, N=5, w=FAKE, stream=0)
MATMUL = dict(x=FAKE, dtype=0, ld=64, w=FAKE, M=3, K=64, N=5, y=FAKE, act=0, stream=0)
MOE = dict(x=FAKE, dtype=0, ld=64, T=3, H=64, I=32, E=4, k=2, renorm=1, router=FAKE, gate_up=FAKE, down=FAKE,
           y=FAKE, ids=FAKE, weights=FAKE, stream=0)

NULL, INVALID, UNSUPPORTED, OK = (L.WQBMM_ERR_NULLPTR, L.WQBMM_ERR_INVALID, L.WQBMM_ERR_UNSUPPORTED, L.WQBMM_OK)


def cases(name, args, pointers, empty, more):
    for p in pointers:
        yield name, args, {p: 0}, NULL
        yield name, args, {p: MIS}, INVALID
    yield name, args, {}, OK_FOR_A_GPU
    for over, want in more:
        yield name, args, over, want
    if empty:
        for over in empty:
            yield name, args, over, OK


K_RULES = [({"K": 0}, INVALID), ({"K": -32}, INVALID), ({"K": 48}, INVALID), ({"K": 2 ** 20 + 32}, INVALID),
           ({"K": I64_MAX}, INVALID)]
M_RULES = [({"M": -1}, INVALID), ({"M": 2 ** 24 + 1}, INVALID), ({"M": I64_MAX}, INVALID)]
LD_RULES = [({"ld": 63}, INVALID), ({"ld": 68}, INVALID), ({"ld": 56}, INVALID), ({"ld": -64}, INVALID),
            ({"ld": I64_MAX - 7}, INVALID)]
N_RULES = [({"N": 0}, INVALID), ({"N": -1}, INVALID), ({"N": 2 ** 24 + 1}, INVALID), ({"N": I64_MAX}, INVALID)]
TYPES = [({"dtype": 3}, UNSUPPORTED), ({"dtype": -1}, UNSUPPORTED)]

ALL = [c for group in (
    cases("wqbmm_mxfp4_quantize", QUANTIZE, ["x", "codes", "scales"],
          [{"M": 0}, {"M": 0, "x": 0, "codes": 0, "scales": 0}],
          K_RULES + M_RULES + LD_RULES + TYPES + [({"x": 0, "K": 7}, NULL), ({"K": 48, "dtype": 9}, INVALID)]),
    cases("wqbmm_mxfp4_dequantize", DEQUANTIZE, ["codes", "scales", "y"],
          [{"M": 0}, {"M": 0, "y": 0, "codes": 0, "scales": 0}], K_RULES + M_RULES + LD_RULES + TYPES),
    cases("wqbmm_mxfp4_tile_weights", TILE, ["codes", "scales", "w"], None, K_RULES + N_RULES),
    cases("wqbmm_mxfp4_matmul", MATMUL, ["x", "w", "y"], [{"M": 0}, {"M": 0, "x": 0, "y": 0}],
          K_RULES + M_RULES + LD_RULES + N_RULES + TYPES +
          [({"dtype": 2}, UNSUPPORTED), ({"act": 2}, INVALID), ({"act": -1}, INVALID), ({"M": 0, "w": 0}, NULL)]),
    cases("wqbmm_mxfp4_moe", MOE, ["x", "router", "gate_up", "down", "y", "ids", "weights"],
          [{"T": 0}, {"T": 0, "x": 0, "y": 0, "ids": 0, "weights": 0}],
          LD_RULES + TYPES +
          [({"dtype": 2}, UNSUPPORTED), ({"T": -1}, INVALID), ({"T": 65}, INVALID), ({"H": 48}, INVALID),
           ({"H": 0}, INVALID), ({"I": 0}, INVALID), ({"I": 40}, INVALID), ({"I": I64_MAX}, INVALID),
           ({"E": 0}, INVALID), ({"E": 257}, INVALID), ({"E": I64_MAX}, INVALID), ({"k": 0}, INVALID),
           ({"k": 5}, INVALID), ({"E": 64, "k": 17}, INVALID), ({"E": 256, "I": 2 ** 16}, INVALID),
           ({"E": 256, "H": 2 ** 17, "ld": 2 ** 17}, INVALID), ({"T": 0, "router": 0}, NULL)]),
) for c in group]


@pytest.mark.parametrize("name,args,over,want", ALL, ids=[f"{c[0][12:]}-{c[2]}" for c in ALL])
def test_c_abi_refusals(no_device_visible, name, args, over, want):
    assert call(name, args, over) == want


@pytest.mark.parametrize("K,N,want", [
    (32, 1, 1024 + 256 + 16), (128, 16, 1024 + 256 + 16), (160, 17, 2 * (2 * 1024 + 256) + 16),
    (4096, 4096, 256 * (32 * 1024 + 8 * 256 + 4)),
    (0, 16, -1), (48, 16, -1), (32, 0, -1), (2 ** 20 + 32, 16, -1), (32, 2 ** 24 + 1, -1),
])
def test_tiled_weight_bytes(K, N, want):
    assert L.lib().wqbmm_mxfp4_tiled_weight_bytes(K, N) == want


# ---- refusals of the wrappers ------------------------------------------------------------

def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    import weight_only_quantized_msd_amd as W
    x = torch.zeros(2, 64, dtype=torch.float16)
    codes, scales = torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)
    for f in (lambda: W.wqbmm_mxfp4_quantize(x),
              lambda: W.wqbmm_mxfp4_dequantize(codes, scales, torch.float16),
              lambda: W.wqbmm_mxfp4_tile_weights(codes, scales),
              lambda: W.wqbmm_mxfp4_matmul(x, codes, 2),
              lambda: W.wqbmm_mxfp4_moe(x, x, codes, codes, 32, 1)):
        with pytest.raises(ValueError, match="device tensor"):
            f()
