"""The operators that train what stands around the experts, where a general formula takes a value of its own: no rows
with weights that are not finite, expert windows, scores at the end of fp32's range, confident rows. Tolerances as in
test_block_gradients_gpu, which hold for the router kernels' exponentials too: these are off by 2^-22 + |v| (2^-24 + 2^-26)
of themselves, 2^-18.7 at the |v| <= 30 that a share of p above 2^-43 has, beside sums of at most 37 terms (2^-18.8)."""
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


@pytest.mark.parametrize("T,E,k", [(9, 17, 3), (40, 128, 4), (333, 256, 8), (70, 1024, 32)])
def test_rows_of_faint_scores_keep_their_quotients(moe, T, E, k):
    """Sigmoid scores far below 1 in every expert, down to where the router's own fp32 score is 0 (a logit of -88.7),
    and softmax scores that a bias chose from the far end: what is divided by their sum stays what it is."""
    g = gen(T + E)
    for low in (-16.9, -17.5, -40.0, -84.0):
        x = low - 4 * torch.rand(T, E, generator=g)
        ids = torch.argsort(torch.rand(T, E, generator=g), 1)[:, :k].int()
        ids[T // 2] = -1
        off = [0, T // 3, T - 1]
        check_balance(moe, x, ids, "sigmoid", off)
        for renorm in (True, False):
            if renorm or low > -60:
                check_router_backward(moe, x, ids, "sigmoid", renorm, off)
    # one row of each kind beside the others
    x = 3 * torch.randn(T, E, generator=g)
    x[::2] -= 90 - x[::2].amax(1, keepdim=True).neg() - 8
    x[::2] = torch.minimum(x[::2], torch.tensor(-70.0))
    x[::2, 0] = -82.0
    check_balance(moe, x, ids, "sigmoid")
    check_router_backward(moe, x, ids, "sigmoid", True)
    # chosen experts 50 to 95 below a row's largest logit
    x = torch.randn(T, E, generator=g)
    far = torch.argsort(torch.rand(T, E - 1, generator=g), 1)[:, :min(k, E - 1)] + 1
    x[:, 0] = 1.0
    x.scatter_(1, far, -50 - 45 * torch.rand(T, 1, generator=g) + torch.randn(T, far.shape[1], generator=g))
    check_router_backward(moe, x, far.int(), "softmax", True)
    check_router_backward(moe, x, far.int(), "softmax", True, losses=False)


def test_gradient_of_weights_of_faint_scores_that_a_bias_chose(moe):
    """Through router_scored: where its weights are normalised and not 0, so are the gradient's."""
    for scoring, x in (("sigmoid", -86 + torch.rand(6, 32, generator=gen(1))),
                       ("softmax", torch.cat((torch.full((6, 1), 80.0), torch.rand(6, 31, generator=gen(2)) * 2), 1))):
        bias = torch.zeros(32)
        bias[5:20] = 2.0
        dw = torch.randn(6, 4, generator=gen(3))
        ids, w = moe.router_scored(x.cuda(), 4, scoring, bias.cuda(), route_scale=2.5)
        assert (w > 0).all() and torch.allclose(w.sum(1), torch.full((6,), 2.5).cuda())
        got = f64(moe.router_backward(x.cuda(), ids, dw.cuda(), scoring, route_scale=2.5))
        ref, mag = P.router_backward(x.numpy(), ids.cpu().numpy(), f64(dw), scoring, True, 2.5)
        assert np.all(np.abs(got - ref) <= 2.0 ** -16 * mag) and np.abs(got).max() > 0.05


def test_scores_that_the_router_has_as_0(moe):
    """Logits below -88.8, or a chosen softmax score below fp32's least: no weights, no gradient, no share of p."""
    x = torch.full((2, 8), -90.0)
    x[1] = -89.0
    ids = torch.tensor([[1, 2], [3, 4]], dtype=torch.int32)
    b = moe.router_balance(x.cuda(), ids.cuda(), "sigmoid")
    assert not b.prob.any() and float(b.stats[2]) == 2
    g = moe.router_backward(x.cuda(), ids.cuda(), torch.ones(2, 2).cuda(), "sigmoid", stats=b.stats, slope=b.slope,
                            grad_losses=torch.tensor([1.0, 0.0]).cuda())
    assert not g.any()
    x = torch.zeros(1, 8)
    x[0, 1:3] = torch.tensor([-106.0, -107.0])
    assert not moe.router_backward(x.cuda(), ids[:1].cuda(), torch.tensor([[1.0, 2.0]]).cuda(), "softmax").any()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_z_loss_of_confident_rows(moe, scoring):
    """One logit of 0 and others far below: log(1 + d), d the others' exponentials. d is off by 2^-20 of itself, 1 + d
    by half a step of 2^-23, the logarithm by 2^-23 of itself; z is its square."""
    a = np.linspace(2.0, 15.0, 53).astype(np.float32)
    for E in (2, 8):
        for many in (False, True):
            x = torch.full((len(a), E), -INF)
            x[:, 0] = 0
            x[:, E - 1] = -torch.from_numpy(a)
            ids = torch.zeros(len(a), 1, dtype=torch.int32)
            off = torch.arange(len(a) + 1, dtype=torch.int32)
            d = np.exp(-a.astype(np.float64))
            lse = np.log1p(d)
            e = 2.0 ** -20 * d + 2.0 ** -24 + 2.0 ** -23 * lse
            if many:
                z = f64(moe.router_balance(x.cuda(), ids.cuda(), scoring, off.cuda()).stats[1])
                assert abs(z - np.mean(lse ** 2)) <= np.mean(2 * lse * e + e * e) + 2.0 ** -20 * np.mean(lse ** 2)
                continue
            for t in range(len(a)):
                b = moe.router_balance(x[t:t + 1].cuda(), ids[:1].cuda(), scoring)
                assert abs(float(b.stats[1]) - lse[t] ** 2) <= 2 * lse[t] * e[t] + e[t] ** 2 + 2.0 ** -22 * lse[t] ** 2
                g = f64(moe.router_backward(x[t:t + 1].cuda(), ids[:1].cuda(), None, scoring, stats=b.stats, slope=b.slope,
                                            grad_losses=torch.tensor([0.0, 1.0]).cuda()))[0]
                want = 2 * lse[t] / (1 + d[t]) * np.array([1.0, d[t]])
                tol = 2 * e[t] / (1 + d[t]) * np.array([1.0, d[t]]) + 2.0 ** -19 * want
                assert np.all(np.abs(g[[0, E - 1]] - want) <= tol)
