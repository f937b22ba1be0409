"""The operators that train what stands around the experts, where a general formula takes a value of its own: no rows
with weights that are not finite, expert windows, scores at the end of fp32's range, confident rows. Tolerances as in
test_block_gradients_gpu."""
import numpy as np
import pytest
import torch

from oracle import operators_oracle as P
from test_block_gradients_gpu import check_balance, check_router_backward, f64, gen, moe  # noqa: F401

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_no_rows_and_weights_that_are_not_finite(moe, bad):
    """A sum over no rows is 0, whatever factors it would have had."""
    K = 96
    e = torch.empty(0, K, dtype=torch.bfloat16, device="cuda")
    w = torch.full((K,), bad, dtype=torch.bfloat16, device="cuda")
    for act in ("linear", "sigmoid"):
        r = moe.sandwich_norm_backward(e, e, e, e, torch.empty(2, 0, device="cuda"), w, w, w[None].clone(), act, e,
                                       torch.full((1,), bad, device="cuda"))
        for t in (r.post_gamma, r.pre_gamma, r.gate, r.residual_scale):
            assert torch.equal(t, torch.zeros_like(t))
