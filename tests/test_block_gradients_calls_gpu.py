"""Calls of the operators that train what stands around the experts, as their documentation allows and refuses them."""
import pytest
import torch

from test_block_gradients_gpu import cuda, gen, make_backward, moe, rows, same  # noqa: F401

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


@pytest.mark.parametrize("K,act,ck", [(96, "linear", None), (2880, "sigmoid", "ocp"), (8224, "sigmoid", None)])
def test_gate_for_every_value_of_a_batch_of_one(moe, K, act, ck):
    """gate_per "value" keeps the gate's meaning, its gradient's type and every bit with one row as with more."""
    d = rows(2, K, K, "full")
    one = {n: v[1:].clone() if n in ("x", "residual", "gate") else v for n, v in d.items()}
    both, last = ({n: cuda(v) for n, v in t.items()} for t in (d, one))
    kw = dict(gate_act=act, gate_per="value", rstd=True, checkpoint8=ck)
    a, b = moe.sandwich_norm(**both, **kw), moe.sandwich_norm(**last, **kw)
    assert same(a.h[1:], b.h) and same(a.y[1:], b.y) and same(a.rstd[:, 1:], b.rstd)
    call, _ = make_backward(d, act, ck=ck, seed=K)
    cut = lambda n, v: v if not isinstance(v, torch.Tensor) else v[:, 1:].contiguous().cuda() if n == "rstd" \
        else v[1:].clone().cuda() if v.dim() == 2 else v.cuda()
    g2 = moe.sandwich_norm_backward(**{n: cut("", v) if isinstance(v, str) else cuda(v) for n, v in call.items()},
                                    gate_per="value")
    g1 = moe.sandwich_norm_backward(**{n: cut(n, v) for n, v in call.items()}, gate_per="value")
    assert g1.gate.dtype == torch.bfloat16 and g1.gate.shape == (1, K)
    assert same(g2.gate[1:], g1.gate) and same(g2.x[1:], g1.x) and same(g2.residual[1:], g1.residual)
    # without it, and as a channel's: fp32 of the gate's shape
    for per in (None, "channel"):
        c = moe.sandwich_norm_backward(**{n: cut(n, v) for n, v in call.items()}, gate_per=per)
        assert c.gate.dtype == torch.float32 and torch.allclose(c.gate, g1.gate.float(), rtol=2.0 ** -7, atol=1e-6)


def test_gate_per_and_its_refusals(moe):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    x, tok = bf(4, 64), torch.zeros(4, 1, device="cuda")
    for per, gate in (("value", x), ("channel", bf(1, 64)), ("token", tok)):
        a, b = moe.sandwich_norm(x, x, gate=gate), moe.sandwich_norm(x, x, gate=gate, gate_per=per)
        assert same(a.h, b.h)
    for per, gate in (("value", bf(1, 64)), ("value", tok), ("channel", x), ("channel", None), ("token", x),
                      ("token", torch.zeros(1, 1, device="cuda")), ("row", x), ("value", x.cpu())):
        with pytest.raises((ValueError, TypeError)):
            moe.sandwich_norm(x, x, gate=gate, gate_per=per)
        with pytest.raises((ValueError, TypeError)):
            moe.sandwich_norm_backward(x, None, x, None, None, gate=gate, gate_per=per)
