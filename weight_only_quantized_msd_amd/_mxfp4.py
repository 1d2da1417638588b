"""Python wrappers of the MXFP4 operators (C ABI: include/wqbmm_mxfp4.h).

They check tensor metadata, allocate outputs and pass device pointers and the
HIP stream; everything else happens in the kernels.  The calls are short
(several run in a few microseconds), so the wrappers do as little as they can.

Format: 32 consecutive values along the last dimension share a scale byte s
that stands for 2^(s - 127) (255: NaN); two 4-bit elements to a byte, the lower
index in the low nibble.
"""
from __future__ import annotations

from . import _lib
from ._lib import WQBMM_ERR_INVALID, check, lib

_ACTS = {"16bit": _lib.WQBMM_MXFP4_ACT_16BIT, "mxfp4": _lib.WQBMM_MXFP4_ACT_MXFP4}
_dtypes = None


def _dtype_code(dtype, allow_fp32):
    global _dtypes
    if _dtypes is None:
        import torch
        _dtypes = {torch.float16: _lib.WQBMM_DTYPE_F16, torch.bfloat16: _lib.WQBMM_DTYPE_BF16,
                   torch.float32: _lib.WQBMM_DTYPE_F32}
    code = _dtypes.get(dtype)
    if code is None or (code == _lib.WQBMM_DTYPE_F32 and not allow_fp32):
        raise TypeError(f"unsupported type {dtype}: float16 or bfloat16" + (" or float32" if allow_fp32 else ""))
    return code


def _rows(t, name):
    """Checks a 2-D device tensor with contiguous rows; returns (rows, columns, row distance)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    rows, cols = t.shape
    ld, step = t.stride()
    if rows <= 1:            # the distance between rows means nothing then
        ld = (cols + 7) // 8 * 8
    if step != 1 and cols > 1:
        raise ValueError(f"the rows of {name} must be contiguous (any distance between rows that is a multiple of 8)")
    return rows, cols, ld


def _bytes(t, shape, name, device):
    import torch
    if t.dtype != torch.uint8 or t.device != device or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous uint8 tensor of shape {tuple(shape)} on {device}")


def _output(t, shape, dtype, name, device):
    if t.dtype != dtype or t.device != device or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


class _On:
    """The device of the tensors and the stream of the call as the current ones,
    so that outputs are allocated for the stream that writes them."""

    def __init__(self, device, stream):
        import torch
        self._device = torch.cuda.device(device) if torch.cuda.current_device() != device.index else None
        self._stream = torch.cuda.stream(stream) if stream is not None else None

    def __enter__(self):
        import torch
        if self._device:
            self._device.__enter__()
        if self._stream:
            self._stream.__enter__()
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        if self._stream:
            self._stream.__exit__(*exc)
        if self._device:
            self._device.__exit__(*exc)
        return False


def wqbmm_mxfp4_quantize(x, codes=None, scales=None, stream=None):
    """x [M][K] (float16, bfloat16 or float32, K % 32 == 0, rows any multiple of
    8 values apart) -> (codes uint8 [M][K/2], scales uint8 [M][K/32]).

    Per block of 32: 2^(floor(log2(max|x|)) - 2) is the scale; values are
    divided by it, rounded half to even and clipped at 6.  A block with an
    infinity or a NaN reads back as NaN."""
    import torch
    M, K, ld = _rows(x, "x")
    code = _dtype_code(x.dtype, True)
    with _On(x.device, stream) as s:
        if codes is None:
            codes = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
        else:
            _bytes(codes, (M, K // 2), "codes", x.device)
        if scales is None:
            scales = torch.empty((M, K // 32), dtype=torch.uint8, device=x.device)
        else:
            _bytes(scales, (M, K // 32), "scales", x.device)
        check(lib().wqbmm_mxfp4_quantize(x.data_ptr(), code, M, K, ld, codes.data_ptr(), scales.data_ptr(), s),
              "wqbmm_mxfp4_quantize")
    return codes, scales


def wqbmm_mxfp4_dequantize(codes, scales, dtype, y=None, stream=None):
    """codes [M][K/2], scales [M][K/32] -> y [M][K] of `dtype`; y may be given
    (rows any multiple of 8 values apart)."""
    import torch
    if codes.dim() != 2:
        raise ValueError("codes must be a 2-D tensor")
    M, K = codes.shape[0], codes.shape[1] * 2
    code = _dtype_code(dtype, True)
    if not codes.is_cuda:
        raise ValueError("codes must be a device tensor")
    _bytes(codes, (M, K // 2), "codes", codes.device)
    _bytes(scales, (M, K // 32), "scales", codes.device)
    with _On(codes.device, stream) as s:
        if y is None:
            y, ld = torch.empty((M, K), dtype=dtype, device=codes.device), K
        else:
            rows, cols, ld = _rows(y, "y")
            if (rows, cols) != (M, K) or y.dtype != dtype or y.device != codes.device:
                raise ValueError(f"y must be a {dtype} tensor of shape {(M, K)} on {codes.device}")
        check(lib().wqbmm_mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(), M, K, y.data_ptr(), code, ld, s),
              "wqbmm_mxfp4_dequantize")
    return y


def wqbmm_mxfp4_tile_weights(codes, scales, stream=None):
    """One-time layout of a weight W [N][K] (codes [N][K/2], scales [N][K/32]),
    or of a stack of them [E][N][...] with N % 16 == 0; returns uint8
    [wqbmm_mxfp4_tiled_weight_bytes(K, rows)]."""
    import torch
    if codes.dim() not in (2, 3) or not codes.is_cuda:
        raise ValueError("codes must be a device tensor [N][K/2] or [E][N][K/2]")
    *rows, half = codes.shape
    K = half * 2
    _bytes(codes, (*rows, half), "codes", codes.device)
    _bytes(scales, (*rows, K // 32), "scales", codes.device)
    if len(rows) == 2 and rows[1] % 16 != 0:
        raise ValueError("a stack of weights needs N % 16 == 0")
    N = rows[0] * rows[1] if len(rows) == 2 else rows[0]
    nbytes = lib().wqbmm_mxfp4_tiled_weight_bytes(K, N)
    if nbytes < 0:
        check(WQBMM_ERR_INVALID, "wqbmm_mxfp4_tiled_weight_bytes")
    with _On(codes.device, stream) as s:
        w = torch.empty(nbytes, dtype=torch.uint8, device=codes.device)
        check(lib().wqbmm_mxfp4_tile_weights(codes.data_ptr(), scales.data_ptr(), K, N, w.data_ptr(), s),
              "wqbmm_mxfp4_tile_weights")
    return w


def _check_tiled(w, K, N, name, device):
    import torch
    nbytes = lib().wqbmm_mxfp4_tiled_weight_bytes(K, N)
    if nbytes < 0:
        check(WQBMM_ERR_INVALID, "wqbmm_mxfp4_tiled_weight_bytes")
    if w.dtype != torch.uint8 or w.device != device or w.dim() != 1 or w.numel() != nbytes or not w.is_contiguous():
        raise ValueError(f"{name} must be the wqbmm_mxfp4_tile_weights output for {N} rows of {K} on {device}")


def wqbmm_mxfp4_matmul(x, w_tiled, N: int, activations: str = "16bit", y=None, stream=None):
    """y [M][N] = x [M][K] . W^T for a tiled W [N][K]; x and y float16 or
    bfloat16, sums in fp32.  activations "16bit": x as it is; "mxfp4": x is
    quantised (as wqbmm_mxfp4_quantize does) in the call."""
    import torch
    M, K, ld = _rows(x, "x")
    code = _dtype_code(x.dtype, False)
    act = _ACTS.get(activations)
    if act is None:
        raise ValueError(f'activations must be "16bit" or "mxfp4", not {activations!r}')
    _check_tiled(w_tiled, K, N, "w_tiled", x.device)
    with _On(x.device, stream) as s:
        if y is None:
            y = torch.empty((M, N), dtype=x.dtype, device=x.device)
        else:
            _output(y, (M, N), x.dtype, "y", x.device)
        check(lib().wqbmm_mxfp4_matmul(x.data_ptr(), code, ld, w_tiled.data_ptr(), M, K, N, y.data_ptr(), act, s),
              "wqbmm_mxfp4_matmul")
    return y


def wqbmm_mxfp4_moe(x, router, gate_up, down, intermediate: int, top_k: int, renormalize: bool = True, y=None,
                    stream=None):
    """A mixture-of-experts layer for up to 64 tokens; returns (y [T][H], ids
    int32 [T][top_k], weights float32 [T][top_k]).

    x [T][H] and router [E][H] float16 or bfloat16; gate_up: the tiled stack
    [E][2*intermediate][H] (gate rows, then up rows); down: the tiled stack
    [E][H][intermediate].  Per token the top_k experts by router logit (ties
    to the lowest index), their softmax probabilities (divided by their sum if
    renormalize), and the weighted sum of down . (silu(gate . x) * (up . x))."""
    import torch
    T, H, ld = _rows(x, "x")
    code = _dtype_code(x.dtype, False)
    if router.dim() != 2 or router.shape[1] != H:
        raise ValueError("router must be [E][H]")
    E = router.shape[0]
    _output(router, (E, H), x.dtype, "router", x.device)
    _check_tiled(gate_up, H, E * 2 * intermediate, "gate_up", x.device)
    _check_tiled(down, intermediate, E * H, "down", x.device)
    with _On(x.device, stream) as s:
        if y is None:
            y = torch.empty((T, H), dtype=x.dtype, device=x.device)
        else:
            _output(y, (T, H), x.dtype, "y", x.device)
        ids = torch.empty((T, max(top_k, 0)), dtype=torch.int32, device=x.device)
        weights = torch.empty((T, max(top_k, 0)), dtype=torch.float32, device=x.device)
        check(lib().wqbmm_mxfp4_moe(x.data_ptr(), code, ld, T, H, intermediate, E, top_k, 1 if renormalize else 0,
                                    router.data_ptr(), gate_up.data_ptr(), down.data_ptr(), y.data_ptr(),
                                    ids.data_ptr(), weights.data_ptr(), s),
              "wqbmm_mxfp4_moe")
    return y, ids, weights
