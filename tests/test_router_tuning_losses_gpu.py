"""The losses' way into the gate's gradient in examples/router_tuning.py: by themselves, and beside a task's gradient
of like size, against the float64 oracle on the step's own logits."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import operators_oracle as P
from test_block_gradients_gpu import f64

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def R():
    import __graft_entry__
    __graft_entry__.build()
    import router_tuning
    return router_tuning


@pytest.mark.parametrize("T", [7, 70, 400])
@pytest.mark.parametrize("task", [0.0, 0.1])
def test_losses_reach_the_gate(R, T, task):
    """The router's gradient is within 2^-16 of its terms' magnitudes; the step hands on its own weights' gradient,
    stats, slope and offsets, each of which moves it by far more. The gate's is a product over T rows: T + 1
    roundings of 2^-24 of its magnitudes beside the logits' error."""
    K, E, k = 256, 16, 4
    p = R.Layer.random(K=K, I=128, E=E, topk=k, seed=T)
    g = torch.Generator().manual_seed(T)
    x, res, dh, dz = (torch.randn(T, K, generator=g).bfloat16() for _ in range(4))
    off = [0, T // 3, T // 3, T - 1]
    _, _, kept = R.forward(p, x.cuda(), res.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda"))
    logits, ids = f64(kept[3]), kept[4].cpu().numpy()
    bal = P.router_balance(logits, ids, "sigmoid", off)
    # coefficients that give both losses and the task gradients of like size
    for n, coef in enumerate(([1.0, 0.0], [0.0, 1.0], [1.0, 0.5])):
        p.losses = torch.tensor(coef, device="cuda") * T
        got = R.backward(p, kept, (task * dh).cuda(), (task * dz).cuda())
        dw = f64(got["weights"])
        assert bool(np.any(dw)) == (task > 0)
        dl = f64(p.losses)
        ref, mag = P.router_backward(logits, ids, dw, "sigmoid", True, p.route_scale, dl, bal)
        d = f64(got["logits"])
        assert np.all(np.abs(d - ref) <= 2.0 ** -16 * mag + 2.0 ** -126)
        alone = P.router_backward(logits, ids, None, "sigmoid", True, p.route_scale, dl, bal)[0]
        assert np.linalg.norm(alone) > 0.02 * np.linalg.norm(ref) and not d[T - 1].any() == (task == 0)
        want = ref.T @ f64(x)
        tol = (2.0 ** -16 * mag + (T + 1) * 2.0 ** -24 * np.abs(d)).T @ np.abs(f64(x))
        assert np.all(np.abs(f64(got["gate"]) - want) <= tol)
