"""Every form of the norms' gradient in mixed types and with scratch of exactly the size asked for. Tolerances as in
test_block_gradients_gpu."""
import pytest
import torch

from test_block_gradients_gpu import check_backward, cuda, make_backward, moe, rows  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [640, 8224])
@pytest.mark.parametrize("gate,act", [(None, "linear"), ("channel", "linear"), ("channel", "sigmoid"), ("token", "sigmoid"),
                                      ("full", "linear"), ("full", "sigmoid")])
@pytest.mark.parametrize("side", ["x", "h"])
def test_one_side_in_8_bits(moe, K, gate, act, side):
    """x in 8 bits beside a bf16 h, and the other way round; with the residual's scale and without."""
    for T, scaled in ((3, True), (330, False)):
        a, va = make_backward(rows(T, K, 5, gate, scaled=scaled), act)
        b, vb = make_backward(rows(T, K, 5, gate, scaled=scaled), act, ck="ocp")
        a[side], a[side + "_scale"], va[side] = b[side], b[side + "_scale"], vb[side]
        check_backward(moe, a, va)


@pytest.mark.parametrize("T", [1, 2, 3, 76, 153])
@pytest.mark.parametrize("K", [32, 2880, 8224, 16384])
@pytest.mark.parametrize("gate,ck", [("full", None), ("channel", "ocp")])
def test_scratch_of_the_size_asked_for(moe, T, K, gate, ck):
    """The column sums and the scalars of few rows fill the scratch to its end: nothing is written past it."""
    call, vals = make_backward(rows(T, K, T + K, gate), "sigmoid", ck=ck)
    call = {k: v if isinstance(v, str) else cuda(v) for k, v in call.items()}
    n, G = moe.sandwich_norm_backward_workspace_size(T, K), 4096
    buf = torch.full((n + 2 * G,), 0xA5, dtype=torch.uint8, device="cuda")
    check_backward(moe, call, vals, workspace=buf[G:G + n])
    assert (buf[:G] == 0xA5).all() and (buf[G + n:] == 0xA5).all()


@pytest.mark.parametrize("T,E,S", [(1, 1, 1), (3, 300, 3), (65, 256, 1), (64, 256, 2), (400, 33, 401), (5000, 1024, 7)])
def test_scratch_of_the_losses(moe, T, E, S):
    x = torch.randn(T, E, device="cuda")
    ids = torch.randint(0, E, (T, 1), dtype=torch.int32, device="cuda")
    off = torch.linspace(0, T, S + 1, device="cuda").int()
    n, G = moe.router_balance_workspace_size(T, E, S), 4096
    buf = torch.full((n + 2 * G,), 0xA5, dtype=torch.uint8, device="cuda")
    r = moe.router_balance(x, ids, "softmax", off, workspace=buf[G:G + n])
    assert int(r.counts.sum()) == T
    assert (buf[:G] == 0xA5).all() and (buf[G + n:] == 0xA5).all()
