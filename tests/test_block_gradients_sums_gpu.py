"""Sums over all rows in the gradient of the norms around a block, where they cancel."""
import numpy as np
import pytest
import torch

from oracle import operators_oracle as P
from test_block_gradients_gpu import cuda, f64, gen, make_backward, moe, rows  # noqa: F401

pytestmark = pytest.mark.gpu


def signs(T, kind):
    """+-1 a row: of one sign for many rows in a row, for two (a CTA's), one, or at random."""
    t = torch.arange(T)
    if kind == "random":
        return 1 - 2 * torch.randint(0, 2, (T,), generator=gen(T))
    return 1 - 2 * (t // {"halves": (T + 1) // 2, "pairs": 2, "rows": 1}[kind] % 2)


@pytest.mark.parametrize("kind", ["halves", "pairs", "rows", "random"])
@pytest.mark.parametrize("T,K", [(1, 64), (2, 2880), (3, 8224), (300, 2880), (4096, 2880), (777, 16384), (1000, 7168),
                                 (100_003, 64)])
def test_gradient_of_the_residual_scale_is_an_exact_sum(moe, T, K, kind):
    """Without a norm the gradient's terms are grad_h * residual: of whole numbers up to 127 whole numbers below
    2^14, so that every sum and every remainder is a whole number below 2^24 that fp32 holds, a sum's value apart,
    whose remainder is kept: the result is the sum, rounded once."""
    g = gen(T + K)
    dh = signs(T, kind)[:, None] * torch.randint(64, 128, (T, K), generator=g)
    res = torch.randint(64, 128, (T, K), generator=g)
    want = np.float32(int((dh * res).sum()))
    x = torch.randn(T, K, generator=g).bfloat16()
    kw = dict(residual=res.bfloat16().cuda(), residual_scale=torch.ones(1, device="cuda"))
    full = torch.randn(T, K, generator=g).bfloat16().cuda()
    x8 = dict(x=torch.randn(T, K, generator=g).to(torch.float8_e4m3fn).cuda(),
              x_scale=torch.full((T, K // 32), 127, dtype=torch.uint8, device="cuda"))
    for a in (dict(x=x.cuda()), x8):
        for gate in ({}, dict(gate=full), dict(gate=full, gate_act="sigmoid"), dict(gate=full[:1].clone())):
            r = moe.sandwich_norm_backward(dh.bfloat16().cuda(), None, h=None, rstd=None, **a, **gate, **kw)
            assert float(r.residual_scale) == want, (gate.keys(), float(r.residual_scale), want)


@pytest.mark.parametrize("gate,ck", [("full", None), ("token", "nosat")])
def test_gradient_of_the_residual_scale_of_a_cancelling_sum(moe, gate, ck):
    """The whole formula. Its terms d * residual are off by d's two roundings, at most 2^-24 of d each and independent:
    with probability one but for 1e-14 by at most 8 sqrt(2) 2^-24 of the root of the terms' squares. A row's mean(v H)
    passes 13 additions, 8 in a thread and 5 in trees or more: 8 sqrt(13) 2^-24 < 2^-19 of its terms' root, the
    same for all values of the row."""
    for seed in range(6):
        d = rows(777, 2880, 100 + seed, gate)
        call, v = make_backward(d, "sigmoid", ck=ck, seed=seed)
        got = float(moe.sandwich_norm_backward(**{k: t if isinstance(t, str) else cuda(t) for k, t in call.items()})
                    .residual_scale)
        ref = P.sandwich_norm_backward(**v)
        terms = ref["residual"] / v["scale"] * v["residual"]
        H, vy = v["h"] * v["r2"][:, None], v["dy"] * v["pre_gamma"]
        row = v["r2"] * np.sqrt(np.sum((vy * H) ** 2, 1)) / H.shape[1] * np.abs(np.sum(H * v["residual"], 1))
        tol = 2.0 ** -24 * (8 * 2 ** 0.5 * np.sqrt(np.sum(terms ** 2)) + abs(got)) + 2.0 ** -19 * np.sqrt(np.sum(row ** 2))
        assert abs(got - ref["residual_scale"]) <= tol, (seed, got, ref["residual_scale"], tol)


def test_gradient_of_the_residual_scale_out_of_range(moe):
    """A sum past fp32's range is infinite and a NaN a NaN, remainders or not."""
    x = torch.ones(40, 64, dtype=torch.bfloat16, device="cuda")
    kw = dict(x=x, h=None, rstd=None, residual_scale=torch.ones(1, device="cuda"))
    big = torch.full_like(x, 1e38)
    for gate in (None, x):
        run = lambda dh, res: float(moe.sandwich_norm_backward(dh, None, residual=res, gate=gate, **kw).residual_scale)
        assert run(big, x) == float("inf") and run(-big, x) == -float("inf")
        bad = x.clone()
        bad[39, 63] = float("nan")
        assert np.isnan(run(bad, x)) and np.isnan(run(x, bad))
        bad[39, 63] = float("inf")
        assert run(bad, x) == float("inf") and run(x, -bad) == -float("inf")


@pytest.mark.parametrize("gate", [None, "channel", "full"])
@pytest.mark.parametrize("ck", [None, "ocp"])
def test_gradient_of_the_residual_scale_with_values_that_are_not_finite(moe, gate, ck):
    """An infinite residual beside a finite kept h: its term's sign. A NaN of h makes its row NaN."""
    call, v = make_backward(rows(20, 96, 3, gate), "linear", ck=ck, seed=4)
    run = lambda: float(moe.sandwich_norm_backward(**{k: t if isinstance(t, str) else cuda(t) for k, t in call.items()})
                        .residual_scale)
    sign = np.sign(P.sandwich_norm_backward(**v)["residual"] / v["scale"])
    for at in ((0, 0), (7, 50), (19, 95)):
        keep = call["residual"]
        for big in (float("inf"), -float("inf"), float("nan")):
            call["residual"] = keep.clone()
            call["residual"][at] = big
            got = run()
            assert got == sign[at] * big or (np.isnan(big) and np.isnan(got))
        call["residual"] = keep
    if ck is None:
        call["h"][7, 50] = float("nan")
    else:
        call["h_scale"][7, 1] = 255
    assert np.isnan(run())
