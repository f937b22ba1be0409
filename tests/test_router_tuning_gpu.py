"""The operators around the experts run together, as in examples/router_tuning.py: one forward and backward step
against float64 differentiation of the whole chain, with the experts' outputs, the choice of experts and the counts
held fixed (as the step itself holds them)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.fixture(scope="module")
def R():
    import __graft_entry__
    __graft_entry__.build()
    import router_tuning
    return router_tuning


def inputs(T, K, seed):
    g = torch.Generator().manual_seed(seed)
    t = [torch.randn(T, K, generator=g).bfloat16() for _ in range(4)]
    off = torch.tensor([0, T // 3, T // 3, T - 1], dtype=torch.int32)     # an empty sequence, a row in none
    return t[0], t[1], t[2] * 0.1, t[3] * 0.1, off


@pytest.mark.parametrize("T", [1, 7, 70])
def test_step_against_float64_differentiation(R, T):
    """Tolerance, in the norm of each gradient: the kept activations' MXFP8 codes are off by at most half a step,
    2^-4 relative (2^-4 / sqrt(3) in root mean square, both x and h), each of which enters a gradient once, plus
    bf16 roundings of the layer's output and of the gradients handed on (2^-8 each, four of them): 0.036 * 2 + 0.016,
    under 0.09."""
    K, I, E, k = 256, 128, 16, 4
    p = R.Layer.random(K=K, I=I, E=E, topk=k, seed=T)
    x, res, dh, dz, off = inputs(T, K, T)
    h, z, kept = R.forward(p, x.cuda(), res.cuda(), off.cuda())
    got = R.backward(p, kept, dh.cuda(), dz.cuda())
    torch.cuda.synchronize()
    ids, w, balance, routes = kept[4].cpu().long(), kept[5], kept[6], kept[7]
    d = lambda t: t.detach().double().cpu()
    leaf = {n: d(getattr(p, n)).requires_grad_(True) for n in ("gate", "post", "pre", "channel", "scale")}
    r = d(res).requires_grad_(True)
    logits = d(x) @ leaf["gate"].t()
    logits.retain_grad()
    s = torch.sigmoid(logits)
    wt = s.gather(1, ids)
    wt = wt / wt.sum(-1, keepdim=True) * p.route_scale
    wt.retain_grad()
    y = (wt[:, :, None] * d(routes).view(T, k, K)).sum(1)
    n = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-5) * leaf["post"]
    hh = leaf["scale"] * r + leaf["channel"] * n
    zz = hh / torch.sqrt((hh * hh).mean(-1, keepdim=True) + 1e-5) * leaf["pre"]
    prob = s / s.sum(-1, keepdim=True)
    losses, tokens = [], 0
    zl = torch.zeros((), dtype=torch.float64)
    o = off.tolist()
    for a, b in zip(o[:-1], o[1:]):
        if b > a:
            share = E * torch.bincount(ids[a:b].flatten(), minlength=E).double() / ((b - a) * k)
            losses.append((share * prob[a:b].mean(0)).sum())
            zl = zl + torch.logsumexp(logits[a:b], -1).square().sum()
            tokens += b - a
    c = d(p.losses)
    total = (hh * d(dh)).sum() + (zz * d(dz)).sum()
    if losses:
        total = total + c[0] * sum(losses) / len(losses) + c[1] * zl / tokens
        assert abs(float(balance.stats[0]) - float(sum(losses) / len(losses))) <= 1e-5
        assert float(balance.stats[2]) == tokens and float(balance.stats[3]) == len(losses)
    total.backward()
    want = {n: t.grad for n, t in leaf.items()}
    want.update(residual=r.grad, logits=logits.grad, weights=wt.grad)
    # outputs: bf16 of the layer's y and of the result
    for a, b in ((h, hh), (z, zz)):
        assert float((d(a) - b.detach()).norm()) <= 2e-2 * float(b.detach().norm())
    for name, g in got.items():
        a, b = d(g), want[name].reshape(g.shape)
        if name == "scale":      # a sum that cancels: against the magnitudes of its terms
            ref = float((r.grad / leaf["scale"].detach()).abs().mul(d(res).abs()).sum())
        else:
            ref = float(b.norm())
        assert float((a - b).norm()) <= 0.09 * ref + 1e-12, (name, float((a - b).norm()), ref)


def test_step_captured_twice_and_replayed(R):
    """Two graphs of the step on the same inputs, replayed in turn, give the eager step's bits."""
    p = R.Layer.random(K=512, I=128, E=32, topk=4, seed=3)
    x, res, dh, dz, off = (t.cuda() for t in inputs(300, 512, 5))

    def step():
        h, z, kept = R.forward(p, x, res, off)
        return [h, z, *R.backward(p, kept, dh, dz).values()]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
    side.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(out, want):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_example_runs(R):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "router_tuning.py"), "--tokens", "64", "--steps", "2"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "us a step" in r.stdout
