"""Tuning what stands around an MXFP4 layer whose experts stay as they are: the router's gate, the norms after and
before the block and the block's gate for each channel. One step, forward and backward, through the library:

    logits  = x @ gate.T
    ids, w  = router on the logits                                    router_scored
    stats   = balance losses and expert counts, sequence by sequence  router_balance
    y, o    = routed experts, and each route's own output             forward, forward_window
    h, z    = residual + channel gate * norm(y), normed for the next  sandwich_norm (x and h kept in 8 bits)

    dy, ... = gradients of the norms and the channel gate             sandwich_norm_backward
    dw      = gradient of the routing weights                         combine_backward
    dlogits = gradient of the weights and of both losses              router_backward
    dgate   = dlogits.T @ x

Usage: python examples/router_tuning.py [--tokens T] [--steps N]   (one GB300)
runs N steps captured in a CUDA graph and prints the time of one and the balance losses.
"""
from __future__ import annotations

import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mxfp4_mixture_experts_gb300 import moe  # noqa: E402


@dataclasses.dataclass
class Layer:
    """Frozen experts and the parameters that are tuned."""
    w13: torch.Tensor
    s13: torch.Tensor
    w2: torch.Tensor
    s2: torch.Tensor
    gate: torch.Tensor       # fp32 [E, K]
    bias: torch.Tensor       # fp32 [E], the balance bias (steers the choice, has no gradient)
    post: torch.Tensor       # bf16 [K]
    pre: torch.Tensor        # bf16 [K]
    channel: torch.Tensor    # bf16 [1, K]
    scale: torch.Tensor      # fp32 [1], of the residual
    losses: torch.Tensor     # fp32 [2], coefficients of the balance and the z loss
    topk: int = 8
    route_scale: float = 2.5

    @staticmethod
    def random(K=2048, I=1024, E=64, topk=8, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
        u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.uint8)
        return Layer(u8(0, 256, E, 2 * I, K // 2), u8(112, 118, E, 2 * I, K // 32), u8(0, 256, E, K, I // 2),
                     u8(112, 118, E, K, I // 32), rn(E, K) / K ** 0.5, 0.05 * rn(E), (0.5 + 0.1 * rn(K)).bfloat16(),
                     (1 + 0.1 * rn(K)).bfloat16(), (0.8 + 0.1 * rn(1, K)).bfloat16(),
                     torch.full((1,), 0.9, device="cuda"), torch.tensor([1e-2, 1e-3], device="cuda"), topk)


def forward(p: Layer, x, residual, offsets):
    """x bf16 [T, K], the layer's normed input, residual bf16 [T, K], offsets int32 [S + 1] of the
    sequences -> the new residual stream, its normed rows, and what the backward pass needs."""
    logits = x.float() @ p.gate.t()
    ids, w = moe.router_scored(logits, p.topk, "sigmoid", p.bias, route_scale=p.route_scale)
    balance = moe.router_balance(logits, ids, "sigmoid", offsets)
    y = moe.forward(x, ids, w, p.w13, p.s13, p.w2, p.s2)
    routes = moe.forward_window(x, ids, None, p.w13, p.s13, p.w2, p.s2, per_route=True)
    norm = moe.sandwich_norm(y, residual, p.post, p.pre, gate=p.channel, residual_scale=p.scale, checkpoint8="nosat",
                             rstd=True)
    return norm.h, norm.y, (x, residual, offsets, logits, ids, w, balance, routes, norm)


def backward(p: Layer, kept, grad_h, grad_z):
    """Gradients of a loss with grad_h and grad_z (bf16 [T, K]) at the outputs plus p.losses times the
    balance and the z loss: dict of gate, post, pre, channel, scale, residual, logits and weights."""
    x, residual, offsets, logits, ids, w, balance, routes, norm = kept
    g = moe.sandwich_norm_backward(grad_h, grad_z, norm.x8, norm.h8, norm.rstd, p.post, p.pre, gate=p.channel,
                                   residual=residual, residual_scale=p.scale, x_scale=norm.x8_scale,
                                   h_scale=norm.h8_scale)
    dw, _ = moe.combine_backward(g.x, routes, ids, w)
    dlogits = moe.router_backward(logits, ids, dw, "sigmoid", route_scale=p.route_scale, grad_losses=p.losses,
                                  stats=balance.stats, slope=balance.slope, seq_offsets=offsets)
    return dict(gate=dlogits.t() @ x.float(), post=g.post_gamma, pre=g.pre_gamma, channel=g.gate,
                scale=g.residual_scale, residual=g.residual, logits=dlogits, weights=dw)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    args = ap.parse_args()
    p = Layer.random()
    T, K = args.tokens, p.post.shape[0]
    g = torch.Generator(device="cuda").manual_seed(1)
    x, residual, dh, dz = (torch.randn(T, K, generator=g, device="cuda").bfloat16() for _ in range(4))
    offsets = torch.tensor([0, T // 3, T // 2, T], dtype=torch.int32, device="cuda")

    def step():
        _, _, kept = forward(p, x, residual, offsets)
        # the balance losses alone drive the gate here: no task gradient
        grads = backward(p, kept, dh * 0, dz * 0)
        p.gate -= 50.0 * grads["gate"]
        return kept[6].stats

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        print("balance and z loss before:", step()[:2].tolist())
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stats = step()
    start, end = torch.cuda.Event(True), torch.cuda.Event(True)
    start.record()
    for _ in range(args.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{T} tokens: {1e3 * start.elapsed_time(end) / args.steps:.0f} us a step; losses after: {stats[:2].tolist()}")


if __name__ == "__main__":
    main()
