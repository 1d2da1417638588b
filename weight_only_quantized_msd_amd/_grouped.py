"""Python wrappers of the operators whose weights depend on the row (C ABI:
include/wqbmm_grouped.h): the choice of experts, the order of rows by group,
grouped products with MXFP4 weights, the weighted sum of a token's experts, and
low-rank adapters beside a shared projection.

As in _mxfp4.py the ordinary call is made in C++ (csrc/mx_torch.cpp) and what that
hands back undone takes the way below, which also says what is wrong with a call;
the calls have no gradients, and a backward pass that reaches one raises.

A plan, (offsets, rows), says which rows belong to which group; it is made and
stays on the device.  A mixture-of-experts layer for any number of tokens:

    ids, weights = wqbmm_moe_route(logits, top_k)
    offsets, rows, slots = wqbmm_group_rows(ids, experts)
    h = wqbmm_mxfp4_grouped_matmul(x, gate_up, offsets, 2 * intermediate, rows=rows, gated=True)
    z = wqbmm_mxfp4_grouped_matmul(h, down, offsets, hidden)
    y = wqbmm_moe_combine(z, slots, weights)
"""
from __future__ import annotations

from . import _mxfp4 as _m
from ._lib import check, lib


def _matrix(t, name):
    """Checks a 2-D device tensor with contiguous rows, any distance of at least their length apart; (rows,
    columns, row distance)."""
    rows, cols, ld = _m._rows(t, name)
    if ld < cols:            # expanded, or overlapping windows: the kernels count on rows of their own
        raise ValueError(f"the rows of {name} must not overlap")
    return rows, cols, ld


def _index(t, dims, name, device):
    if t.dtype != _m._torch.int32 or t.device != device or t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dims}-D int32 tensor on {device}")


def _pointer(t):
    return None if t is None else t.data_ptr()


def wqbmm_moe_route(logits, top_k: int, renormalize: bool = True, stream=None):
    """logits [T][E] (float32, float16 or bfloat16) -> (ids int32 [T][top_k], weights
    float32 [T][top_k]): per token the top_k experts with the largest logits (ties to
    the lowest index), in descending order, and their softmax probabilities (divided by
    their sum if renormalize).  An expert whose logit is -inf is not chosen; where
    fewer than top_k are left the ids are -1 and the weights 0."""
    torch = _m._torch or _m._load()
    if stream is None:
        both = _m._calls.moe_route(logits, top_k, renormalize)
        if both is not None:
            return both
    T, E, ld = _matrix(logits, "logits")
    code = _m._dtype_code(logits.dtype, True)

    def work(s):
        ids = logits.new_empty((T, max(top_k, 0)), dtype=torch.int32)
        weights = logits.new_empty((T, max(top_k, 0)), dtype=torch.float32)
        check(lib().wqbmm_moe_route(logits.data_ptr(), code, ld, T, E, top_k, 1 if renormalize else 0, ids.data_ptr(),
                                    weights.data_ptr(), s), "wqbmm_moe_route")
        return ids, weights

    return _m._with_history("wqbmm_moe_route", _m._on(logits.device, stream, work), logits)


def wqbmm_group_rows(ids, groups: int, stream=None):
    """Choices ids (int32 [T][k], or [T]) of `groups` groups -> the plan (offsets int32
    [groups + 1], rows int32 [T*k], slots like ids): the choices ordered by group,
    those of a group by token.  Group g has the places offsets[g] to offsets[g + 1] - 1,
    rows says which token a place stands for, slots the place of each choice.  An id
    outside [0, groups) is a choice of no group: its place is behind the last group's,
    its slot -1."""
    torch = _m._torch or _m._load()
    if stream is None:
        plan = _m._calls.group_rows(ids, groups)
        if plan is not None:
            return plan
    if not ids.is_cuda:
        raise ValueError("ids must be a device tensor")
    if ids.dim() not in (1, 2):
        raise ValueError("ids must be [T][k] or [T]")
    _index(ids, ids.dim(), "ids", ids.device)
    T, k = ids.shape if ids.dim() == 2 else (ids.shape[0], 1)

    def work(s):
        offsets = ids.new_empty(max(groups, 0) + 1)
        rows, slots = ids.new_empty(T * k), torch.empty_like(ids)
        check(lib().wqbmm_group_rows(ids.data_ptr(), T, k, groups, offsets.data_ptr(), rows.data_ptr(),
                                     slots.data_ptr(), s), "wqbmm_group_rows")
        return offsets, rows, slots

    return _m._on(ids.device, stream, work)


def wqbmm_mxfp4_grouped_matmul(x, w_tiled, offsets, N: int, rows=None, activations: str = "16bit",
                               gated: bool = False, y=None, stream=None):
    """Products of groups of rows with a weight each: y [S][N], y[s] = W_g . x[rows[s]] for
    the places s of group g (offsets [G + 1]; rows [S], or None: x's rows are the places).

    x [R][K] float16 or bfloat16; w_tiled: the tiled stack [G][N][K], N % 16 == 0;
    activations as for wqbmm_mxfp4_matmul.  gated: W_g has N / 2 gate rows, then N / 2 up
    rows, and y [S][N / 2] is silu(gate . x) * (up . x).  Places of no group are not
    written (allocated here, they hold anything); a place whose row lies outside x gets
    zeros."""
    _m._torch or _m._load()
    act = _m._ACTS.get(activations)
    if act is None:
        raise ValueError(f'activations must be "16bit" or "mxfp4", not {activations!r}')
    if stream is None:
        out = _m._calls.grouped_matmul(x, w_tiled, offsets, N, rows, act, gated, y)
        if out is not None:
            return out
    R, K, ld = _m._rows(x, "x")
    code = _m._dtype_code(x.dtype, False)
    device = x.device
    _index(offsets, 1, "offsets", device)
    if rows is not None:
        _index(rows, 1, "rows", device)
    G, S = offsets.shape[0] - 1, R if rows is None else rows.shape[0]
    if G < 1:
        raise ValueError("offsets must be [G + 1]")
    _m._check_tiled(w_tiled, K, G * N, "w_tiled", device)
    _m._refuse_given_output(y, "wqbmm_mxfp4_grouped_matmul", x)
    n_out = N // 2 if gated else N
    if y is not None:
        _m._exactly(y, (S, n_out), x.dtype, "y", device)

    def work(s):
        out = x.new_empty((S, n_out)) if y is None else y
        check(lib().wqbmm_mxfp4_grouped_matmul(x.data_ptr(), code, ld, R, _pointer(rows), offsets.data_ptr(), G, S, K,
                                               N, w_tiled.data_ptr(), out.data_ptr(), act, 1 if gated else 0, s),
              "wqbmm_mxfp4_grouped_matmul")
        return out

    return _m._with_history("wqbmm_mxfp4_grouped_matmul", (_m._on(device, stream, work),), x)[0]


def _of_shape(t, shape, dtype, name, device):
    """Checks a matrix of that shape with contiguous rows; its row distance."""
    rows, cols, ld = _matrix(t, name)
    if (rows, cols) != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {shape} on {device}")
    return ld


def wqbmm_moe_combine(z, slots, weights, base=None, y=None, stream=None):
    """y [T][H] = base + the sum over a token's choices of weights[t][j] * z[slots[t][j]], in
    float32 and in order; slots (int32 [T][k]) outside z's rows add nothing.  z [S][H], base
    and y [T][H] float16 or bfloat16 (rows any multiple of 8 values apart, H % 8 == 0),
    weights float32 [T][k].  y may be base."""
    torch = _m._torch or _m._load()
    if stream is None:
        out = _m._calls.moe_combine(z, slots, weights, base, y)
        if out is not None:
            return out
    S, H, ldz = _matrix(z, "z")
    code = _m._dtype_code(z.dtype, False)
    device = z.device
    _index(slots, 2, "slots", device)
    T, k = slots.shape
    _m._exactly(weights, (T, k), torch.float32, "weights", device)
    ldb = 0 if base is None else _of_shape(base, (T, H), z.dtype, "base", device)
    inputs = [t for t in (z, weights, base) if t is not None]
    _m._refuse_given_output(y, "wqbmm_moe_combine", *inputs)
    ldy = H if y is None else _of_shape(y, (T, H), z.dtype, "y", device)

    def work(s):
        out = z.new_empty((T, H)) if y is None else y
        check(lib().wqbmm_moe_combine(z.data_ptr(), code, ldz, S, H, slots.data_ptr(), weights.data_ptr(), T, k,
                                      _pointer(base), ldb, out.data_ptr(), ldy, s), "wqbmm_moe_combine")
        return out

    return _m._with_history("wqbmm_moe_combine", (_m._on(device, stream, work),), *inputs)[0]


def wqbmm_lora_matmul(x, a, b, offsets, rows, scales=None, base=None, y=None, stream=None):
    """y [M][N] = base + scales[l] * (x . A_l^T) . B_l^T for the rows of adapter l; rows of no
    adapter: base.  base is what a shared projection gives for x (None: 0).

    x [M][K] float16 or bfloat16; a [L][r][K], b [L][N][r] of x's type (r % 8 == 0, at most
    256; smaller adapters padded with zeros); (offsets, rows): the plan
    of wqbmm_group_rows(ids, L) for an id per row, one for all projections of a step;
    scales float32 [L].  y may be base; then rows of no adapter are not touched."""
    torch = _m._torch or _m._load()
    if stream is None:
        out = _m._calls.lora_matmul(x, a, b, offsets, rows, scales, base, y)
        if out is not None:
            return out
    M, K, ldx = _m._rows(x, "x")
    code = _m._dtype_code(x.dtype, False)
    device = x.device
    if a.dim() != 3 or b.dim() != 3 or a.shape[2] != K or b.shape[0] != a.shape[0] or b.shape[2] != a.shape[1]:
        raise ValueError("a must be [L][r][K] and b [L][N][r]")
    (L, r, _), N = a.shape, b.shape[1]
    _m._exactly(a, (L, r, K), x.dtype, "a", device)
    _m._exactly(b, (L, N, r), x.dtype, "b", device)
    _m._exactly(offsets, (L + 1,), torch.int32, "offsets", device)
    _m._exactly(rows, (M,), torch.int32, "rows", device)
    if scales is not None:
        _m._exactly(scales, (L,), torch.float32, "scales", device)
    ldb = 0 if base is None else _of_shape(base, (M, N), x.dtype, "base", device)
    inputs = [t for t in (x, a, b, scales, base) if t is not None]
    _m._refuse_given_output(y, "wqbmm_lora_matmul", *inputs)
    ldy = N if y is None else _of_shape(y, (M, N), x.dtype, "y", device)

    def work(s):
        out = x.new_empty((M, N)) if y is None else y
        check(lib().wqbmm_lora_matmul(x.data_ptr(), code, ldx, M, K, N, r, L, a.data_ptr(), b.data_ptr(),
                                      _pointer(scales), offsets.data_ptr(), rows.data_ptr(), _pointer(base), ldb,
                                      out.data_ptr(), ldy, s), "wqbmm_lora_matmul")
        return out

    return _m._with_history("wqbmm_lora_matmul", (_m._on(device, stream, work),), *inputs)[0]
