"""MXFP4 operators from their definitions, in numpy and 64 bits, and how far a
kernel may be from them.

Error bounds.  u(t) = finfo(t).eps / 2 is half a step of type t relative to the
value (bf16 2^-8, fp16 2^-11); below the smallest normal number the half step
is absolute (`tiny`).  A sum of n products in fp32, in any order, with products
exact, is within n * 2^-23 * sum|products| (2^-24 per rounded addition; twice
that, because the matrix cores may truncate where an addition rounds).
"""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([MAGNITUDES, -MAGNITUDES])

U = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134}      # half the spacing of subnormals
STEP32 = 2.0 ** -23


def nearest_code(a):
    """Magnitude codes 0..7 nearest to a >= 0; a tie goes to the even code; above 6 is 6."""
    a = np.minimum(np.asarray(a, np.float64), 6.0)
    d = np.abs(a[..., None] - MAGNITUDES)
    best = d.min(-1, keepdims=True)
    tied = d == best                                   # one or two neighbours
    first = tied.argmax(-1)
    two = tied.sum(-1) == 2
    return np.where(two & (first % 2 == 1), first + 1, first).astype(np.uint8)


def quantize(x):
    """x [M][K] (any float type) -> (codes uint8 [M][K/2], scales uint8 [M][K/32])."""
    x = np.asarray(x).astype(np.float64)
    M, K = x.shape
    b = x.reshape(M, K // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    safe = np.where(bad[..., None], 0.0, b)
    top = np.abs(safe).max(-1)
    e = np.frexp(top)[1] - 1 - 2                       # floor(log2(top)) - 2
    e = np.where(top == 0, -127, np.clip(e, -127, 127))
    code = nearest_code(np.abs(safe) * 2.0 ** (-e[..., None].astype(np.float64)))
    code = code | (np.signbit(safe).astype(np.uint8) << 3)
    code = np.where(bad[..., None], 0, code).astype(np.uint8).reshape(M, K)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def dequantize(codes, scales):
    """The values in 64 bits [..., K]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return VALUES[c] * np.repeat(s, 32, -1)


def matmul(x, w, dtype):
    """(y, bound) of x [M][K] . w [N][K]^T in 64 bits; `bound`: how far a
    result in `dtype` may be."""
    y = x @ w.T
    slack = x.shape[1] * STEP32 * (np.abs(x) @ np.abs(w).T)
    return y, rounded(y, slack, dtype)


def rounded(y, slack, dtype):
    """slack of the value before it is rounded to `dtype`, plus the rounding."""
    return slack + U[dtype] * (np.abs(y) + slack) + TINY[dtype]


def route(x, router, k, renormalize):
    """(ids, weights, gap, slack): the k largest logits, ties to the lowest
    index; gap: the least distance between a chosen logit and the next one;
    slack: how far an fp32 logit may be off."""
    logits = x @ router.T
    order = np.argsort(-logits, axis=-1, kind="stable")
    ids = order[:, :k]
    chosen = np.take_along_axis(logits, order[:, :min(k + 1, logits.shape[1])], 1)
    gap = np.min(chosen[:, :-1] - chosen[:, 1:]) if chosen.shape[1] > 1 else np.inf
    p = np.exp(logits - logits.max(-1, keepdims=True))
    picked = np.take_along_axis(p, ids, 1)
    weights = picked / (picked if renormalize else p).sum(-1, keepdims=True)
    slack = x.shape[1] * STEP32 * np.max(np.abs(x) @ np.abs(router).T)
    return ids, weights, gap, slack


def moe(x, router, gate_up, down, k, renormalize, dtype):
    """(y, bound, ids, weights, weight_bound, gap, slack) of the layer; the
    weights gate_up [E][2I][H] and down [E][H][I] as values."""
    T, H = x.shape
    E, _, inter = down.shape
    ids, weights, gap, slack = route(x, router, k, renormalize)
    # exp of a logit off by slack, each exp and division a few fp32 steps, a sum of E terms
    weight_rel = 2 * slack * 1.01 + (E + 16) * STEP32
    y, err, mass = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            g, u = np.split(gate_up[e] @ x[t], 2)
            eg, eu = np.split(H * STEP32 * (np.abs(gate_up[e]) @ np.abs(x[t])), 2)
            silu = g / (1 + np.exp(-g))
            # |silu'| < 1.1; exp, 1 + exp and the division: 8 fp32 steps of the value
            es = 1.1 * eg + 8 * STEP32 * np.abs(silu)
            h = silu * u * weights[t, j]
            eh = weights[t, j] * (es * (np.abs(u) + eu) + np.abs(silu) * eu)
            # the weight's own error, two products, and the split into two bf16 parts (2^-16)
            eh += np.abs(h) * (weight_rel + 2 * STEP32 + 2.0 ** -16)
            y[t] += down[e] @ h
            err[t] += np.abs(down[e]) @ eh
            mass[t] += np.abs(down[e]) @ np.abs(h)
    err += (k * inter * 2 + 16) * STEP32 * mass          # two products for each element of h
    return y, rounded(y, err, dtype), ids, weights, weight_rel * weights, gap, slack
