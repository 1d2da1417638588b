"""Python wrappers of the MXFP4 operators (C ABI: include/wqbmm_mxfp4.h).

They check tensor metadata, allocate outputs and pass device pointers and the
HIP stream; everything else happens in the kernels.  The calls are short
(several run in a few microseconds), so the ordinary one, which allocates its
outputs on the current stream of the current device, is made in C++
(csrc/mx_torch.cpp, the module _mx_calls); what that hands back undone takes the
way below, which also says what is wrong with a call.

The calls have no gradients.  What they return for inputs that require one carries
the call in its history, and a backward pass that reaches it raises.

Format: 32 consecutive values along the last dimension share a scale byte s
that stands for 2^(s - 127) (255: NaN); two 4-bit elements to a byte, the lower
index in the low nibble.
"""
from __future__ import annotations

from . import _lib
from ._lib import WQBMM_ERR_INVALID, check, lib

_ACTS = {"16bit": _lib.WQBMM_MXFP4_ACT_16BIT, "mxfp4": _lib.WQBMM_MXFP4_ACT_MXFP4}
_torch = None            # torch and what is looked up in it once, set by _load
_calls = None            # csrc/mx_torch.cpp
_end_of_history = None   # an autograd function without a backward pass
_dtypes = {}
_device_now = _raw_stream = None


class _TheOtherWay:
    """_mx_calls that hands every call back."""
    quantize = dequantize = matmul = moe = staticmethod(lambda *args: None)


def _load():
    global _torch, _device_now, _raw_stream, _calls, _end_of_history
    import torch
    lib()
    if _lib.OTHER_LIB:                      # _mx_calls would load the package's own beside it
        _mx_calls = _TheOtherWay
    else:
        try:
            from . import _mx_calls
        except ImportError as e:
            raise RuntimeError("_mx_calls.so is not built; "
                               "run `python -c 'import __graft_entry__ as g; g.build()'`") from e
    _dtypes.update({torch.float16: _lib.WQBMM_DTYPE_F16, torch.bfloat16: _lib.WQBMM_DTYPE_BF16,
                    torch.float32: _lib.WQBMM_DTYPE_F32})
    _device_now, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _torch, _calls = torch, _mx_calls

    class EndOfHistory(torch.autograd.Function):
        @staticmethod
        def forward(ctx, where, outputs, *inputs):
            ctx.where = where
            ctx.mark_non_differentiable(*[t for t in outputs if not t.is_floating_point()])
            return tuple(outputs)

        @staticmethod
        def backward(ctx, *gradients):
            raise RuntimeError(f"{ctx.where} has no gradient")

    _end_of_history = EndOfHistory
    return torch


def _needs_gradient(*inputs):
    return _torch.is_grad_enabled() and any(t.requires_grad for t in inputs)


def _refuse_given_output(y, where, *inputs):
    if y is not None and _needs_gradient(y, *inputs):
        raise RuntimeError(f"{where} has no gradient: with y given, its inputs and y must not require one")


def _with_history(where, outputs, *inputs):
    """outputs, with a history that ends in an error if an input requires a gradient."""
    return _end_of_history.apply(where, outputs, *inputs) if _needs_gradient(*inputs) else outputs


def _dtype_code(dtype, allow_fp32):
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


def _exactly(t, shape, dtype, name, device):
    if t.dtype != dtype or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _on(device, stream, work):
    """work(raw stream) with the tensors' device and the call's stream as the
    current ones, so that outputs are allocated for the stream that writes them."""
    if stream is None:
        if _device_now() == device.index:
            return work(_raw_stream(device.index))
        with _torch.cuda.device(device):
            return work(_raw_stream(device.index))
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    with _torch.cuda.stream(stream):
        return work(stream.cuda_stream)


def wqbmm_mxfp4_quantize(x, codes=None, scales=None, stream=None):
    """x [M][K] (float16, bfloat16 or float32, K % 32 == 0, rows any multiple of
    8 values apart) -> (codes uint8 [M][K/2], scales uint8 [M][K/32]).

    Per block of 32: 2^(floor(log2(max|x|)) - 2) is the scale; values are
    divided by it, rounded half to even and clipped at 6.  A block with an
    infinity or a NaN reads back as NaN."""
    torch = _torch or _load()
    if codes is None and scales is None and stream is None:
        both = _calls.quantize(x)
        if both is not None:
            return both
    M, K, ld = _rows(x, "x")
    code = _dtype_code(x.dtype, True)
    device = x.device
    if codes is not None:
        _exactly(codes, (M, K // 2), torch.uint8, "codes", device)
    if scales is not None:
        _exactly(scales, (M, K // 32), torch.uint8, "scales", device)

    def work(s):
        c = x.new_empty((M, K // 2), dtype=torch.uint8) if codes is None else codes
        e = x.new_empty((M, K // 32), dtype=torch.uint8) if scales is None else scales
        check(lib().wqbmm_mxfp4_quantize(x.data_ptr(), code, M, K, ld, c.data_ptr(), e.data_ptr(), s),
              "wqbmm_mxfp4_quantize")
        return c, e

    return _on(device, stream, work)


def wqbmm_mxfp4_dequantize(codes, scales, dtype, y=None, stream=None):
    """codes [M][K/2], scales [M][K/32] -> y [M][K] of `dtype`; y may be given
    (rows any multiple of 8 values apart)."""
    torch = _torch or _load()
    if y is None and stream is None:
        out = _calls.dequantize(codes, scales, _dtype_code(dtype, True))
        if out is not None:
            return out
    if not codes.is_cuda:
        raise ValueError("codes must be a device tensor")
    if codes.dim() != 2:
        raise ValueError("codes must be a 2-D tensor")
    M, half = codes.shape
    K, ld = half * 2, half * 2
    code = _dtype_code(dtype, True)
    device = codes.device
    _exactly(codes, (M, half), torch.uint8, "codes", device)
    _exactly(scales, (M, K // 32), torch.uint8, "scales", device)
    if y is not None:
        rows, cols, ld = _rows(y, "y")
        if (rows, cols) != (M, K) or y.dtype != dtype or y.device != device:
            raise ValueError(f"y must be a {dtype} tensor of shape {(M, K)} on {device}")

    def work(s):
        out = codes.new_empty((M, K), dtype=dtype) if y is None else y
        check(lib().wqbmm_mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(), M, K, out.data_ptr(), code, ld, s),
              "wqbmm_mxfp4_dequantize")
        return out

    return _on(device, stream, work)


def wqbmm_mxfp4_tile_weights(codes, scales, stream=None):
    """One-time layout of a weight W [N][K] (codes [N][K/2], scales [N][K/32]),
    or of a stack of them [E][N][...] with N % 16 == 0; returns uint8
    [wqbmm_mxfp4_tiled_weight_bytes(K, rows)]."""
    torch = _torch or _load()
    if codes.dim() not in (2, 3) or not codes.is_cuda:
        raise ValueError("codes must be a device tensor [N][K/2] or [E][N][K/2]")
    *rows, half = codes.shape
    K = half * 2
    _exactly(codes, (*rows, half), torch.uint8, "codes", codes.device)
    _exactly(scales, (*rows, K // 32), torch.uint8, "scales", codes.device)
    if len(rows) == 2 and rows[1] % 16 != 0:
        raise ValueError("a stack of weights needs N % 16 == 0")
    N = rows[0] * rows[1] if len(rows) == 2 else rows[0]
    nbytes = _tiled_bytes(K, N)

    def work(s):
        w = codes.new_empty(nbytes)
        check(lib().wqbmm_mxfp4_tile_weights(codes.data_ptr(), scales.data_ptr(), K, N, w.data_ptr(), s),
              "wqbmm_mxfp4_tile_weights")
        return w

    return _on(codes.device, stream, work)


def _tiled_bytes(K, N):
    nbytes = lib().wqbmm_mxfp4_tiled_weight_bytes(K, N)
    if nbytes < 0:
        check(WQBMM_ERR_INVALID, "wqbmm_mxfp4_tiled_weight_bytes")
    return nbytes


def _check_tiled(w, K, N, name, device):
    if (w.dtype != _torch.uint8 or w.device != device or w.dim() != 1 or w.numel() != _tiled_bytes(K, N)
            or not w.is_contiguous()):
        raise ValueError(f"{name} must be the wqbmm_mxfp4_tile_weights output for {N} rows of {K} on {device}")


def wqbmm_mxfp4_matmul(x, w_tiled, N: int, activations: str = "16bit", y=None, stream=None):
    """y [M][N] = x [M][K] . W^T for a tiled W [N][K]; x and y float16 or
    bfloat16, sums in fp32.  activations "16bit": x as it is; "mxfp4": x is
    quantised (as wqbmm_mxfp4_quantize does) in the call."""
    _torch or _load()
    act = _ACTS.get(activations)
    if act is None:
        raise ValueError(f'activations must be "16bit" or "mxfp4", not {activations!r}')
    if y is None and stream is None:
        out = _calls.matmul(x, w_tiled, N, act)
        if out is not None:
            return out
    M, K, ld = _rows(x, "x")
    code = _dtype_code(x.dtype, False)
    device = x.device
    _check_tiled(w_tiled, K, N, "w_tiled", device)
    _refuse_given_output(y, "wqbmm_mxfp4_matmul", x)
    if y is not None:
        _exactly(y, (M, N), x.dtype, "y", device)

    def work(s):
        out = x.new_empty((M, N)) if y is None else y
        check(lib().wqbmm_mxfp4_matmul(x.data_ptr(), code, ld, w_tiled.data_ptr(), M, K, N, out.data_ptr(), act, s),
              "wqbmm_mxfp4_matmul")
        return out

    return _with_history("wqbmm_mxfp4_matmul", (_on(device, stream, work),), x)[0]


def wqbmm_mxfp4_moe(x, router, gate_up, down, intermediate: int, top_k: int, renormalize: bool = True, y=None,
                    stream=None):
    """A mixture-of-experts layer for up to 64 tokens; returns (y [T][H], ids
    int32 [T][top_k], weights float32 [T][top_k]).

    x [T][H] and router [E][H] float16 or bfloat16; gate_up: the tiled stack
    [E][2*intermediate][H] (gate rows, then up rows); down: the tiled stack
    [E][H][intermediate].  Per token the top_k experts by router logit (ties
    to the lowest index), their softmax probabilities (divided by their sum if
    renormalize), and the weighted sum of down . (silu(gate . x) * (up . x))."""
    torch = _torch or _load()
    if y is None and stream is None:
        out = _calls.moe(x, router, gate_up, down, intermediate, top_k, renormalize)
        if out is not None:
            return out
    T, H, ld = _rows(x, "x")
    code = _dtype_code(x.dtype, False)
    device = x.device
    if router.dim() != 2 or router.shape[1] != H:
        raise ValueError("router must be [E][H]")
    E = router.shape[0]
    _exactly(router, (E, H), x.dtype, "router", device)
    _check_tiled(gate_up, H, E * 2 * intermediate, "gate_up", device)
    _check_tiled(down, intermediate, E * H, "down", device)
    _refuse_given_output(y, "wqbmm_mxfp4_moe", x, router)
    if y is not None:
        _exactly(y, (T, H), x.dtype, "y", device)

    def work(s):
        out = x.new_empty((T, H)) if y is None else y
        ids = x.new_empty((T, max(top_k, 0)), dtype=torch.int32)
        weights = x.new_empty((T, max(top_k, 0)), dtype=torch.float32)
        check(lib().wqbmm_mxfp4_moe(x.data_ptr(), code, ld, T, H, intermediate, E, top_k, 1 if renormalize else 0,
                                    router.data_ptr(), gate_up.data_ptr(), down.data_ptr(), out.data_ptr(),
                                    ids.data_ptr(), weights.data_ptr(), s),
              "wqbmm_mxfp4_moe")
        return out, ids, weights

    return _with_history("wqbmm_mxfp4_moe", _on(device, stream, work), x, router)
