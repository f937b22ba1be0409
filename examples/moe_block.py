"""One transformer block's MoE half and the next layer's input projection, with every
operator of the library in its place:

    h, x   = residual + attention output, normed          add_rmsnorm
    ids, w = router on the gate's logits                   router_scored
    y      = routed MXFP4 experts                          forward
    h, q   = residual + y, normed, in MXFP8                add_rmsnorm(out8=...)
    out    = MXFP4 projection + each request's adapter     linear

Usage: python examples/moe_block.py [--tokens T] [--adapters L]   (one GB300)
prints the time of a block captured in a CUDA graph.
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
class Block:
    """Weights of the block, random, in the layouts that the library reads."""
    gamma1: torch.Tensor     # bf16 [K]
    gate: torch.Tensor       # fp32 [E, K]
    bias: torch.Tensor       # fp32 [E], the balance bias
    w13: torch.Tensor
    s13: torch.Tensor
    w2: torch.Tensor
    s2: torch.Tensor
    gamma2: torch.Tensor     # bf16 [K]
    w: torch.Tensor          # uint8 [N, K/2]
    s: torch.Tensor          # uint8 [N, K/32]
    a: torch.Tensor          # bf16 [L, rank, K]
    b: torch.Tensor          # bf16 [L, N, rank]
    scale: torch.Tensor      # fp32 [L]
    topk: int = 8
    n_group: int = 8
    topk_group: int = 4
    route_scale: float = 2.5

    @staticmethod
    def random(K=2048, I=1024, E=64, N=3584, L=16, rank=16, topk=8, n_group=8, topk_group=4, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
        u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.uint8)
        return Block((1 + 0.1 * rn(K)).bfloat16(), rn(E, K) / K ** 0.5, 0.05 * rn(E),
                     u8(0, 256, E, 2 * I, K // 2), u8(112, 118, E, 2 * I, K // 32),
                     u8(0, 256, E, K, I // 2), u8(112, 118, E, K, I // 32),
                     (1 + 0.1 * rn(K)).bfloat16(), u8(0, 256, N, K // 2), u8(114, 120, N, K // 32),
                     (rn(L, rank, K) / K ** 0.5).bfloat16(), (0.1 * rn(L, N, rank)).bfloat16(),
                     1 + torch.rand(L, generator=g, device="cuda"), topk, n_group, topk_group)


def block(p: Block, attn: torch.Tensor, residual: torch.Tensor, adapter_ids: torch.Tensor):
    """attn, residual bf16 [T, K], adapter_ids int32 [T] -> the next projection's output bf16
    [T, N], the residual stream and the chosen experts."""
    x, h, _, _ = moe.add_rmsnorm(attn, p.gamma1, residual)
    logits = x.float() @ p.gate.t()
    ids, w = moe.router_scored(logits, p.topk, "sigmoid", p.bias, p.n_group, p.topk_group,
                               route_scale=p.route_scale)
    y = moe.forward(x, ids, w, p.w13, p.s13, p.w2, p.s2)
    _, h, q, sq = moe.add_rmsnorm(y, p.gamma2, h, out8="nosat", bf16=False)
    out = moe.linear(q, p.w, p.s, sq, adapter_ids=adapter_ids, adapter_a=p.a, adapter_b=p.b,
                     adapter_scale=p.scale)
    return out, h, ids


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--adapters", type=int, default=16)
    args = ap.parse_args()
    p = Block.random(L=args.adapters)
    K = p.gamma1.shape[0]
    g = torch.Generator(device="cuda").manual_seed(1)
    attn = torch.randn(args.tokens, K, generator=g, device="cuda").bfloat16()
    residual = (4 * torch.randn(args.tokens, K, generator=g, device="cuda")).bfloat16()
    # one request a token, some without an adapter
    ids = torch.randint(-1, args.adapters, (args.tokens,), generator=g, device="cuda", dtype=torch.int32)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block(p, attn, residual, ids)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _, chosen = block(p, attn, residual, ids)
    for _ in range(3):
        graph.replay()
    start, end = torch.cuda.Event(True), torch.cuda.Event(True)
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{args.tokens} tokens: {10 * start.elapsed_time(end):.1f} us a block, output rms "
          f"{float(out.float().square().mean().sqrt()):.3f}, {int(chosen.unique().numel())} experts touched")


if __name__ == "__main__":
    main()
