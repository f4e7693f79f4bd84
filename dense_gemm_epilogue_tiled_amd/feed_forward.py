"""A transformer's feed-forward blocks: for decoding, on the operators of mx_ops, and a dense one for training, on
those of train_ops.

    python -m dense_gemm_epilogue_tiled_amd.feed_forward [--tokens T]

runs a dense and a mixture-of-experts block with MX fp4 weights for a few
tokens, captured in a graph as a serving loop would replay it, and prints the
time per block.  With --train it runs training steps of a dense bfloat16 block
(forward, backward, update of the weights) and prints the time per step.
"""
from __future__ import annotations

import argparse

from . import (gated_act, gated_linear, gated_linear_backward, gemm_mxfp4, linear, linear_backward, linear_mxfp4, moe_mxfp4,
               moe_route, mx_quantize, orthogonalize, rms_norm, sandwich_norm, sandwich_norm_backward)


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


# ---- training ---------------------------------------------------------------------

def train_forward(x, residual, w13, w2, norm, next_norm, gate=None, act="silu", scale=1.0, eps=1e-6):
    """``((total, normed), kept)`` of a block whose input x is normed already (the previous block's normed):
    y = W2 (act(W1 x) * W3 x), total = residual + scale * gate * RMS norm of y, normed = the next block's input.

    ``w13`` is the stacked W1 and W3 (2I x H), ``w2`` H x I, ``norm`` and ``next_norm`` the norms' H weights, ``gate`` as for
    sandwich_norm; all float16 or bfloat16."""
    h, gu = gated_linear(x, w13, act=act, keep=True)
    y = linear(h, w2)
    out = sandwich_norm(y, residual, norm, next_norm, gate, scale, eps)
    return out, (x, h, gu, y, out[0])


def train_backward(dtotal, dnormed, kept, w13, w2, norm, next_norm, gate=None, act="silu", scale=1.0, eps=1e-6):
    """``(dx, dresidual, grads)`` from the gradients of train_forward's outputs and what it kept; grads by the
    weights' names."""
    x, h, gu, y, total = kept
    dy, dresidual, dnorm, dnext, dgate = sandwich_norm_backward(dtotal, dnormed, y, total, norm, next_norm, gate, scale, eps)
    dh, dw2, _ = linear_backward(dy, h, w2)
    dx, dw13, _ = gated_linear_backward(dh, x, w13, gu, act)
    return dx, dresidual, {"w13": dw13, "w2": dw2, "norm": dnorm, "next_norm": dnext, "gate": dgate}


def update_matrix(weight, grad, momentum, rate, decay=0.95):
    """One step of a matrix along its orthogonalised momentum, in place: ``momentum`` (float32) decays and takes the
    gradient, and the weight moves by ``rate`` (times the root of its sides' ratio if it is taller than wide) along its
    look-ahead's direction."""
    momentum.mul_(decay).add_(grad)
    step = orthogonalize(momentum.mul(decay).add_(grad), scale=max(1.0, weight.shape[0] / weight.shape[1]) ** 0.5)
    return weight.add_(step.to(weight.dtype), alpha=-rate)


def _train_demo(tokens, hidden, inter, steps):
    import torch
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()

    x, residual, target = rand(tokens, hidden), rand(tokens, hidden), rand(tokens, hidden)
    weights = {"w13": rand(2 * inter, hidden, scale=hidden ** -0.5), "w2": rand(hidden, inter, scale=inter ** -0.5),
               "norm": 1 + rand(hidden, scale=0.1), "next_norm": 1 + rand(hidden, scale=0.1), "gate": rand(hidden, scale=0.1)}
    momentum = {n: torch.zeros_like(weights[n], dtype=torch.float32) for n in ("w13", "w2")}
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for step in range(steps):
        if step == min(1, steps - 1):
            start.record()
        (total, normed), kept = train_forward(x, residual, **weights)
        error = total - target  # the gradient of half the squared distance, for the mean over the tokens
        _, _, grads = train_backward(error / tokens, torch.zeros_like(normed), kept, **weights)
        for n, v in grads.items():
            if n in momentum:
                update_matrix(weights[n], v, momentum[n], 0.02)
            else:
                weights[n].add_(v, alpha=-0.1)
    end.record()
    torch.cuda.synchronize()
    print("training, tokens %d, hidden %d, intermediate %d: %.1f us a step, mean squared distance %.4f" % (
        tokens, hidden, inter, start.elapsed_time(end) / max(1, steps - 1) * 1e3, error.float().square().mean()), flush=True)
    return weights, grads


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
    parser.add_argument("--tokens", type=int, help="default: 1, for training 2048")
    parser.add_argument("--hidden", type=int, default=4096)
    parser.add_argument("--intermediate", type=int, default=2048)
    parser.add_argument("--experts", type=int, default=32)
    parser.add_argument("--topk", type=int, default=4)
    parser.add_argument("--train", action="store_true")
    parser.add_argument("--steps", type=int, default=10, help="of training")
    a = parser.parse_args()
    if a.train:
        _train_demo(a.tokens or 2048, a.hidden, a.intermediate, a.steps)
    else:
        _demo(a.tokens or 1, a.hidden, a.intermediate, a.experts, a.topk)
