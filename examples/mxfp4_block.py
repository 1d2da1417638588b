"""A decoding step and a prompt through one block of a transformer whose weights
are MXFP4: attention's projections, a feed-forward layer for the prompt on MXFP4
activations, and a mixture-of-experts layer for the tokens being decoded.

    python examples/mxfp4_block.py [--hidden 1024] [--ffn 2816] [--experts 16] [--top-k 4]

prints, for each product, how far it is from the same product in fp32 on the
unquantised weights (what quantising costs) and on the quantised ones (what the
kernels add), and the time of a step.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import weight_only_quantized_msd_amd as W


class Mxfp4Linear:
    """y = x . weight^T, the weight [N][K] kept in MXFP4."""

    def __init__(self, weight):
        self.n = weight.shape[0]
        codes, scales = W.wqbmm_mxfp4_quantize(weight)
        self.read_back = W.wqbmm_mxfp4_dequantize(codes, scales, torch.float32)      # for the comparison below
        self.tiled = W.wqbmm_mxfp4_tile_weights(codes, scales)

    def __call__(self, x, activations="16bit"):
        return W.wqbmm_mxfp4_matmul(x, self.tiled, self.n, activations=activations)


class Mxfp4Experts:
    """The experts of a mixture: gate and up rows [E][2I][H], down [E][H][I]."""

    def __init__(self, gate_up, down):
        self.inter = down.shape[2]
        self.tiled = []
        for stack in (gate_up, down):
            E, n, k = stack.shape
            codes, scales = W.wqbmm_mxfp4_quantize(stack.reshape(E * n, k))
            self.tiled.append(W.wqbmm_mxfp4_tile_weights(codes.view(E, n, k // 2), scales.view(E, n, k // 32)))

    def __call__(self, x, router, top_k):
        return W.wqbmm_mxfp4_moe(x, router, *self.tiled, self.inter, top_k)


def distance(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--ffn", type=int, default=2816)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top-k", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=8, help="tokens in a decoding step, at most 64")
    ap.add_argument("--prompt", type=int, default=300, help="tokens in the prompt")
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    H = a.hidden
    qkv_w, up_w = normal(3 * H, H, scale=H ** -0.5), normal(a.ffn, H, scale=H ** -0.5)
    qkv, up = Mxfp4Linear(qkv_w), Mxfp4Linear(up_w)
    experts = Mxfp4Experts(normal(a.experts, 2 * a.ffn, H, scale=H ** -0.5), normal(a.experts, H, a.ffn, scale=a.ffn ** -0.5))
    router = normal(a.experts, H, scale=2 * H ** -0.5)
    prompt, tokens = normal(a.prompt, H), normal(a.tokens, H)

    report = {}
    for name, y, x, layer, weight in (("qkv, decoding", qkv(tokens), tokens, qkv, qkv_w),
                                      ("qkv, prompt", qkv(prompt), prompt, qkv, qkv_w)):
        report[name] = (distance(y, x.float() @ weight.float().t()), distance(y, x.float() @ layer.read_back.t()))
    y = up(prompt, activations="mxfp4")
    x4 = W.wqbmm_mxfp4_dequantize(*W.wqbmm_mxfp4_quantize(prompt), torch.float32)
    report["up, prompt in MXFP4"] = (distance(y, prompt.float() @ up_w.float().t()), distance(y, x4 @ up.read_back.t()))
    for name, (cost, added) in report.items():
        print(f"{name:22s} quantising {cost:.3f}, the kernel {added:.1e}")

    def step(x):
        h = qkv(x)[:, :H].contiguous()
        y, ids, weights = experts(h, router, a.top_k)
        return y, ids, weights

    y, ids, weights = step(tokens)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(50):
        step(tokens)
    end.record()
    end.synchronize()
    print(f"decoding step          {begin.elapsed_time(end) * 20:.1f} us; token 0 goes to experts {ids[0].tolist()}")
    return report, y, ids, weights


if __name__ == "__main__":
    main()
