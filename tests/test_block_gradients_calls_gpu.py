"""Calls of the operators that train what stands around the experts, as their documentation allows and refuses them."""
import pytest
import torch

from test_block_gradients_gpu import gen, moe  # noqa: F401

pytestmark = pytest.mark.gpu


def test_combination_outputs_beside_and_over_inputs(moe):
    """Outputs that end where an input begins and begin where one ends are taken, over one they are refused."""
    T, k, K = 5, 3, 96
    dy, o = torch.randn(T, K, generator=gen(1)).bfloat16().cuda(), torch.randn(T * k, K, generator=gen(2)).bfloat16().cuda()
    w = torch.rand(T, k, generator=gen(3)).cuda()
    want = moe.combine_backward(dy, o, topk_weights=w, routes_too=True)
    n, m = T * K, T * k * K
    buf = torch.full((n + 2 * m,), 7.0, dtype=torch.bfloat16, device="cuda")
    a, b, c = buf[:m].view(T * k, K), buf[m:m + n].view(T, K), buf[m + n:].view(T * k, K)
    for out, ins in ((a, c), (c, a)):
        b.copy_(dy)
        ins.copy_(o)
        got = moe.combine_backward(b, ins, topk_weights=w, grad_routes=out)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[1] is out
        assert torch.equal(b, dy) and torch.equal(ins, o)
    for out in (o, buf[8:8 + m].view(T * k, K), buf[m:m + m].view(T * k, K)):
        with pytest.raises(moe.MoEError):
            moe.combine_backward(b, o if out is o else c, topk_weights=w, grad_routes=out)
