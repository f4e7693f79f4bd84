"""A transformer's feed-forward blocks for decoding, on the operators of mx_ops.

    python -m dense_gemm_epilogue_tiled_amd.feed_forward [--tokens T]

runs a dense and a mixture-of-experts block with MX fp4 weights for a few
tokens, captured in a graph as a serving loop would replay it, and prints the
time per block.
"""
from __future__ import annotations

import argparse

from . import gated_act, gemm_mxfp4, linear_mxfp4, moe_mxfp4, moe_route, mx_quantize, rms_norm


def quantize_weight(w):
    """``(elements, scales)`` of a 16-bit weight (... x N x K) in MX fp4, as the blocks below take it."""
    q, s = mx_quantize(w.reshape(-1, w.shape[-1]), "mxfp4")
    return q.reshape(*w.shape[:-1], -1), s.reshape(*w.shape[:-1], -1)


def dense_block(x, residual, norm, w13, w2, act="silu", eps=1e-6):
    """``(out, total)``: total = x + residual, h = RMS norm of total, out = W2 (act(W1 h) * W3 h).

    ``w13`` and ``w2`` are ``(elements, scales)`` of the stacked W1 and W3 and of W2."""
    h, _, total = rms_norm(x, norm, residual, eps, "same")
    both = linear_mxfp4(h, *w13)
    half = both.shape[1] // 2
    mid, _ = gated_act(both[:, :half], both[:, half:], act, "same")
    return linear_mxfp4(mid, *w2), total


def dense_block_fp4(x, residual, norm, w13, w2, act="silu", eps=1e-6):
    """dense_block with the activations in MX fp4 as well: norm and gated activation write the products' operands."""
    h, scale, total = rms_norm(x, norm, residual, eps, "mxfp4")
    both = gemm_mxfp4(h, scale, *w13, act="none", out_dtype=x.dtype)
    half = both.shape[1] // 2
    mid, scale = gated_act(both[:, :half], both[:, half:], act, "mxfp4")
    return gemm_mxfp4(mid, scale, *w2, act="none", out_dtype=x.dtype), total


def moe_block(x, residual, norm, router, topk, w13, w2, act="silu", eps=1e-6):
    """``(out, total)``: total = x + residual, h = RMS norm of total, out = the topk experts of h by the router."""
    h, _, total = rms_norm(x, norm, residual, eps, "same")
    ids, weights = moe_route(h, router, topk)
    return moe_mxfp4(h, ids, weights, *w13, *w2, act=act), total


def _demo(tokens, hidden, inter, experts, topk):
    import torch
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()

    x, residual, norm = rand(tokens, hidden), rand(tokens, hidden), 1 + rand(hidden, scale=0.1)
    dense = quantize_weight(rand(2 * inter, hidden, scale=0.02)), quantize_weight(rand(hidden, inter, scale=0.02))
    moe = (quantize_weight(rand(experts, 2 * inter, hidden, scale=0.02)),
           quantize_weight(rand(experts, hidden, inter, scale=0.02)))
    router = rand(experts, hidden, scale=2 * hidden ** -0.5)
    blocks = {"dense": lambda: dense_block(x, residual, norm, *dense),
              "dense, fp4 activations": lambda: dense_block_fp4(x, residual, norm, *dense),
              "%d of %d experts" % (topk, experts): lambda: moe_block(x, residual, norm, router, topk, *moe)}
    for name, block in blocks.items():
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            block()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                block()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        graph.replay()
        start.record()
        for _ in range(10):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        print("%-24s tokens %d, hidden %d, intermediate %d: %.1f us" % (
            name, tokens, hidden, inter, start.elapsed_time(end) / 200 * 1e3), flush=True)


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__)
    parser.add_argument("--tokens", type=int, default=1)
    parser.add_argument("--hidden", type=int, default=4096)
    parser.add_argument("--intermediate", type=int, default=2048)
    parser.add_argument("--experts", type=int, default=32)
    parser.add_argument("--topk", type=int, default=4)
    a = parser.parse_args()
    _demo(a.tokens, a.hidden, a.intermediate, a.experts, a.topk)
