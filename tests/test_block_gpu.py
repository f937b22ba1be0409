"""The example block against the float64 oracles of its parts, each fed with what the
library handed to that part (so the parts' own tolerances apply)."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import mxfp4_moe_oracle as O
from oracle import operators_oracle as P

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("T", [1, 7, 40])
def test_example_block(T):
    import __graft_entry__
    __graft_entry__.build()
    import moe_block as B
    from mxfp4_mixture_experts_gb300 import moe
    p = B.Block.random(K=256, I=128, E=16, N=392, L=5, rank=8, topk=2, n_group=4, topk_group=2, seed=T)
    g = torch.Generator().manual_seed(T)
    attn = torch.randn(T, 256, generator=g).bfloat16().cuda()
    res = torch.randn(T, 256, generator=g).bfloat16().cuda()
    ad = torch.randint(-1, 5, (T,), generator=g, dtype=torch.int32).cuda()
    out, h2, ids = B.block(p, attn, res, ad)
    torch.cuda.synchronize()
    bits = lambda t: t.cpu().view(torch.int16).numpy().view(np.uint16)
    f = lambda t: t.float().cpu().numpy().astype(np.float64)
    # the norm, the router on its rows, the experts, the second norm, the projection
    h, x = P.add_rmsnorm(bits(attn), bits(p.gamma1), 1e-5, bits(res))
    xg = moe.add_rmsnorm(attn, p.gamma1, res)[0]
    assert np.linalg.norm(f(xg) - x) <= 3e-3 * np.linalg.norm(x)
    logits = (xg.float() @ p.gate.t()).cpu().numpy()
    rid, rw, key = P.router_scored(logits, 2, "sigmoid", p.bias.cpu().numpy(), 4, 2, route_scale=2.5)
    got = ids.cpu().numpy()
    for t in range(T):   # two experts may trade places within the rounding of their scores
        assert np.all(np.abs(np.sort(key[t])[::-1][:2] - key[t][got[t]]) <= 2.0 ** -19)
    s = P.router_scores(logits, "sigmoid")
    w = np.take_along_axis(s, got, 1)
    w = (2.5 * w / w.sum(1, keepdims=True)).astype(np.float32)
    y = O.forward(bits(xg), got.astype(np.int64), w, p.w13.cpu().numpy(), p.s13.cpu().numpy(),
                  p.w2.cpu().numpy(), p.s2.cpu().numpy())
    yb = torch.from_numpy(y).float().bfloat16()
    hb = torch.from_numpy(h).float().bfloat16()
    want = hb.double().numpy() + y
    assert np.linalg.norm(f(h2) - want) <= 5e-3 * np.linalg.norm(want)   # two bf16 roundings and y's 3e-3
    _, x2 = P.add_rmsnorm(bits(yb), bits(p.gamma2), 1e-5, bits(hb))
    q, sq = P.mx8_encode(x2, "nosat")
    z, _, _ = P.linear(q * np.repeat(np.exp2(sq.astype(np.float64) - 127), 32, 1), p.w.cpu().numpy(),
                       p.s.cpu().numpy(), ad.cpu().numpy(), bits(p.a), bits(p.b), p.scale.cpu().numpy())
    # the library's MXFP8 codes differ from the oracle's where y's bf16 rounding (3e-3
    # in norm) crosses a tie: no more than that error and a code's own step of it
    assert np.linalg.norm(f(out) - z) <= 2e-2 * np.linalg.norm(z)
