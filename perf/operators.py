"""Cases for the microscaled 4-bit (MXFP4) operators: quantising to blocks of 32
values with a shared power of two and reading them back, the product of 16-bit
or MXFP4 activations with MXFP4 weights, and a whole mixture-of-experts layer
with MXFP4 experts for a few tokens.

`run` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, where `own` is true, through
weight_only_quantized_msd_amd.  `exact` computes the same from the definition
in 64 bits.

MXFP4: 32 consecutive values along K share the scale 2^(s - 127), s one byte
(255: the block is NaN); an element is a 4-bit sign, two exponent and one
mantissa bit, one of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, two to a byte with the
lower index in the low nibble.  Quantising takes s - 127 = floor(log2(max|x|))
- 2, divides, rounds half to even and clips at 6.
"""
import math

import torch

own = False

BLOCK = 32
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}


# ---- cases -------------------------------------------------------------------

def _roundtrip(name, M, K, dtype, pad=0):
    return {"name": name, "op": "roundtrip", "M": M, "K": K, "dtype": dtype, "pad": pad}


def _matmul(name, M, K, N, dtype, act, pad=0):
    return {"name": name, "op": "matmul", "M": M, "K": K, "N": N, "dtype": dtype, "act": act, "pad": pad}


def _moe(name, T, H, inter, E, k, dtype, renorm=True):
    return {"name": name, "op": "moe", "T": T, "H": H, "inter": inter, "E": E, "k": k, "dtype": dtype,
            "renorm": renorm}


def listed():
    return [
        # one token's activations, quantised and read back: launch latency
        _roundtrip("roundtrip_m1", 1, 4096, "fp16"),
        # a weight matrix of the FFN shape in fp32, taken out of a wider buffer, an odd number of rows
        _roundtrip("roundtrip_rows_fp32", 4099, 11008, "fp32", pad=64),
        # 16-bit activations: one token of decoding
        _matmul("a16_decode_m1", 1, 4096, 4096, "fp16", "16bit"),
        # a batch of 16 tokens through the FFN's up projection
        _matmul("a16_ffn_up_m16", 16, 4096, 11008, "bf16", "16bit"),
        # a short prompt, sizes that divide into no tile
        _matmul("a16_ragged_m130", 130, 4128, 4099, "bf16", "16bit"),
        # a prompt of 2048 tokens
        _matmul("a16_prefill_m2048", 2048, 4096, 4096, "fp16", "16bit"),
        # MXFP4 activations: the decode batch, the prompt, and the widest projection
        _matmul("a4_ffn_up_m16", 16, 4096, 11008, "fp16", "mxfp4"),
        _matmul("a4_prefill_m2048", 2048, 4096, 4096, "bf16", "mxfp4"),
        _matmul("a4_wide_m2001", 2001, 8192, 28672, "bf16", "mxfp4"),
        # a mixture-of-experts layer: one token, many small experts
        _moe("moe_t1_e64", 1, 2048, 1024, 64, 8, "bf16"),
        # a small batch on odd sizes, softmax weights as they are
        _moe("moe_t33_e12", 33, 1056, 736, 12, 3, "fp16", renorm=False),
        # a decode batch that reaches all of eight FFN-sized experts
        _moe("moe_t16_e8", 16, 4096, 11008, 8, 2, "bf16"),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    dtype = rng.choice(["fp16", "bf16"])
    pad = rng.choice([0, 0, 8, 72])
    op = rng.choice(["roundtrip", "a16", "a4", "moe"])
    if op == "roundtrip":
        K = BLOCK * log(1, 512)
        M = log(1, min(8192, 4099 * 11008 // K))
        c = _roundtrip("", M, K, rng.choice(["fp16", "bf16", "fp32"]), pad)
    elif op in ("a16", "a4"):
        K, N = BLOCK * log(2, 256), log(16, 12288)
        M = log(1, 2048)
        c = _matmul("", M, K, N, dtype, "16bit" if op == "a16" else "mxfp4", pad)
    else:
        E = log(2, 128)
        H, inter = BLOCK * log(4, 128), BLOCK * log(4, 64)
        E = max(2, min(E, 8 * 4096 * 11008 // (H * inter)))
        c = _moe("", log(1, 64), H, inter, E, rng.randint(1, min(8, E)), dtype, rng.random() < 0.5)
    del c["name"]
    return c


# ---- inputs --------------------------------------------------------------------

def _activations(g, M, K, dtype, pad):
    """Normal values with a few channels 20 times as large, as activations have; rows `pad` values apart."""
    x = torch.randn(M, K + pad, generator=g, device="cuda")
    hot = torch.rand(K + pad, generator=g, device="cuda") < 0.01
    x = torch.where(hot, 20.0 * x, x).to(DTYPES[dtype])
    return x[:, :K] if pad else x


def _weights(g, *shape):
    """MXFP4 codes and scales of normal weights with a standard deviation of 1/sqrt(K)."""
    w = torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5
    s, mag, neg = _quantise(w)
    code = (mag | (neg << 3)).to(torch.uint8)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), s.to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}
    if case["op"] == "roundtrip":
        state["x"] = _activations(g, case["M"], case["K"], case["dtype"], case["pad"])
        return state
    if case["op"] == "matmul":
        state["x"] = _activations(g, case["M"], case["K"], case["dtype"], case["pad"])
        state["w"] = _weights(g, case["N"], case["K"])
        kept = ["w"]
    else:
        T, H, inter, E = case["T"], case["H"], case["inter"], case["E"]
        state["x"] = torch.randn(T, H, generator=g, device="cuda").to(DTYPES[case["dtype"]])
        state["router"] = (torch.randn(E, H, generator=g, device="cuda") * 2.0 * H ** -0.5).to(DTYPES[case["dtype"]])
        state["gate_up"] = _weights(g, E, 2 * inter, H)
        state["down"] = _weights(g, E, H, inter)
        kept = ["gate_up", "down"]
    if own:
        # the weights' layout, made once when a model is loaded
        import weight_only_quantized_msd_amd as W
        for name in kept:
            state[name + "_tiled"] = W.wqbmm_mxfp4_tile_weights(*state[name])
    return state


# ---- the plain forms ---------------------------------------------------------------

def _power(s):
    """2^(s - 127) in fp32 from the scale bytes: an exponent field, but for the two ends."""
    s = s.to(torch.int32)
    bits = torch.where(s == 0, 0x00400000, torch.where(s == 255, 0x7FC00000, s << 23))
    return bits.to(torch.int32).view(torch.float32)


def _quantise(x):
    """(scale bytes [..., K/32], magnitude codes 0..7 and signs 0/1 [..., K]) of fp32 values, as int32."""
    b = x.unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1)
    field = top.view(torch.int32) >> 23
    s = torch.where(field == 255, 255, (field - 2).clamp(min=0))
    inverse = torch.where(s == 255, 0, 254 - s).to(torch.int32)
    a = b.abs() * _power(inverse)[..., None]
    mag = ((a > 0.25).to(torch.int32) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return s, mag.flatten(-2), torch.signbit(x).to(torch.int32)


def _values(mag, neg, s):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=mag.device)
    v = table[mag.long()]
    v = torch.where(neg != 0, -v, v)
    return (v.unflatten(-1, (-1, BLOCK)) * _power(s)[..., None]).flatten(-2)


def _read(codes, scales):
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int32)
    return _values(code & 7, code >> 3, scales)


def _fake(x):
    """x in fp32, quantised to MXFP4 and read back."""
    s, mag, neg = _quantise(x)
    return _values(mag, neg, s)


def _plain_moe(state):
    c = state["case"]
    x = state["x"].float()
    # in 64 bits: logits next to each other decide which experts are taken
    logits = state["x"].double() @ state["router"].double().t()
    p = torch.softmax(logits, -1)
    order = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    weight = torch.gather(p, 1, order)
    if c["renorm"]:
        weight = weight / weight.sum(-1, keepdim=True)
    weight = weight.float()
    T, slots = c["T"], c["T"] * c["k"]
    if slots < c["E"]:      # the chosen experts alone, one for each choice
        used = order.flatten()
        share = torch.zeros(T, slots, device=x.device)
        share[torch.arange(T, device=x.device).repeat_interleave(c["k"]), torch.arange(slots, device=x.device)] = weight.flatten()
    else:
        used = torch.arange(c["E"], device=x.device)
        share = torch.zeros(T, c["E"], device=x.device).scatter_(1, order, weight)
    gate_up = _read(state["gate_up"][0][used], state["gate_up"][1][used])
    both = torch.matmul(x, gate_up.flatten(0, 1).t()).unflatten(-1, (used.numel(), -1))     # [T][slot][2I]
    gate, up = both.split(c["inter"], -1)
    h = gate / (1.0 + torch.exp(-gate)) * up * share[..., None]
    down = _read(state["down"][0][used], state["down"][1][used])
    y = torch.bmm(h.transpose(0, 1).contiguous(), down.transpose(1, 2).contiguous()).sum(0)
    return {"y": y.to(state["x"].dtype), "ids": order.to(torch.int32), "weights": weight}


def run(state):
    c = state["case"]
    x = state["x"]
    if own:
        import weight_only_quantized_msd_amd as W
        if c["op"] == "roundtrip":
            codes, scales = W.wqbmm_mxfp4_quantize(x)
            return W.wqbmm_mxfp4_dequantize(codes, scales, x.dtype)
        if c["op"] == "matmul":
            return W.wqbmm_mxfp4_matmul(x, state["w_tiled"], c["N"], activations=c["act"])
        y, ids, weights = W.wqbmm_mxfp4_moe(x, state["router"], state["gate_up_tiled"], state["down_tiled"],
                                            c["inter"], c["k"], renormalize=c["renorm"])
        return {"y": y, "ids": ids, "weights": weights}
    if c["op"] == "roundtrip":
        return _fake(x.float()).to(x.dtype)
    if c["op"] == "matmul":
        a = x.float() if c["act"] == "16bit" else _fake(x.float())
        return torch.matmul(a, _read(*state["w"]).t()).to(x.dtype)
    return _plain_moe(state)


# ---- what a pass cannot do without ------------------------------------------------------

def work(case):
    if case["op"] == "roundtrip":
        n = case["M"] * case["K"]
        return {"bytes": 2 * n * SIZE[case["dtype"]], "flops": 0}
    four = 0.5 + 1.0 / BLOCK            # bytes of one MXFP4 weight with its share of the scale
    if case["op"] == "matmul":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * (M * K + M * N) + four * N * K, "flops": 2 * M * N * K}
    T, H, inter, E, k = (case[n] for n in ("T", "H", "inter", "E", "k"))
    reached = E * (1.0 - (1.0 - k / E) ** T)        # experts that T tokens are expected to reach
    return {"bytes": 4 * T * H + 2 * E * H + reached * 3 * H * inter * four + 8 * T * k,
            "flops": 2 * T * E * H + 2 * T * k * 3 * H * inter}


# ---- the definition in 64 bits --------------------------------------------------------

def _exact_read(codes, scales):
    low, high = codes.to(torch.int64) % 16, codes.to(torch.int64) // 16
    c = torch.stack((low, high), -1).reshape(*codes.shape[:-1], -1)
    e, m = (c % 8) // 2, (c % 2).double()
    v = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.pow(2.0, (e - 1).double()))
    v = v * (1.0 - 2.0 * (c // 8).double())
    return v * torch.repeat_interleave(torch.pow(2.0, scales.double() - 127.0), BLOCK, -1)


def _exact_fake(x):
    x = x.double()
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    top = b.abs().max(-1, keepdim=True).values
    e = torch.frexp(top).exponent.double() - 1.0       # floor(log2(top))
    e = torch.where(top == 0, -127.0, e - 2.0).clamp(-127.0, 127.0)
    a = b / torch.pow(2.0, e)
    step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0)).double()
    q = (torch.round(a / step) * step).clamp(-6.0, 6.0)   # round() takes halves to even
    return (q * torch.pow(2.0, e)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "roundtrip":
        return _exact_fake(x)
    if case["op"] == "matmul":
        return (x if case["act"] == "16bit" else _exact_fake(x)) @ _exact_read(*s["w"]).T
    logits = x @ s["router"].double().T
    ids = torch.argsort(-logits, dim=-1, stable=True)[:, :case["k"]]
    chosen = torch.exp(logits - logits.max(-1, keepdim=True).values)
    total = chosen.sum(-1, keepdim=True)
    chosen = torch.take_along_dim(chosen, ids, 1)
    weights = chosen / (chosen.sum(-1, keepdim=True) if case["renorm"] else total)
    y = torch.zeros_like(x)
    for e in range(case["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        both = x[t] @ _exact_read(s["gate_up"][0][e], s["gate_up"][1][e]).T
        gate, up = both[:, :case["inter"]], both[:, case["inter"]:]
        h = gate * torch.sigmoid(gate) * up
        y[t] += weights[t, j][:, None] * (h @ _exact_read(s["down"][0][e], s["down"][1][e]).T)
    return {"y": y, "ids": None, "weights": weights}
