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


@pytest.mark.parametrize("base", [0, 3, 2 ** 31 - 1])
def test_combination_without_a_window_takes_every_expert(moe, base):
    """n_experts 0 is no window: expert_base then skips nothing; only negative ids are padding."""
    T, k, K = 5, 4, 96
    dy, o = torch.randn(T, K, generator=gen(1)).bfloat16(), torch.randn(T * k, K, generator=gen(2)).bfloat16()
    ids = torch.tensor([0, 1, 2, 3, -1, 4, 2 ** 31 - 1, -2 ** 31, 5, 0] * 2, dtype=torch.int32).view(T, k)
    w = torch.rand(T, k, generator=gen(3))
    want = moe.combine_backward(dy.cuda(), o.cuda(), ids.cuda(), w.cuda(), True)
    dw, do = moe.combine_backward(dy.cuda(), o.cuda(), ids.cuda(), w.cuda(), True, expert_base=base)
    assert torch.equal(dw, want[0]) and torch.equal(do, want[1])
    assert torch.equal(dw.cpu() != 0, ids >= 0)
    ref, _, dref = P.combine_backward(f64(dy), f64(o).reshape(T, k, K), ids.numpy(), f64(w), base)
    assert np.array_equal(ref != 0, ids.numpy() >= 0) and np.abs(f64(dw) - ref).max() <= 1e-4
