"""The operators that train what stands around the experts, where one wrong choice shows: rings that wrap, rows far
from 1, the most rows, infinite logits, long sums. Tolerances as in test_block_gradients_gpu."""
import numpy as np
import pytest
import torch

from oracle import operators_oracle as P
from test_block_gradients_gpu import (check_backward, check_forward, check_router_backward, cuda, f64, gen,
                                      make_backward, moe, rows, same)  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K", [(700, 7168), (330, 16384), (1300, 6144), (650, 8160)])
@pytest.mark.parametrize("gate", [None, "channel", "full"])
def test_long_rows_that_wrap_their_rings(moe, T, K, gate):
    ck = {None: "ocp", "channel": None, "full": "nosat"}[gate]
    d = rows(T, K, T + K, gate, scaled=gate != "channel")
    check_forward(moe, d, "sigmoid", out8="nosat" if K != 16384 else None, ck=ck)
    check_backward(moe, *make_backward(d, "sigmoid", ck=None if K == 16384 and ck else ck, seed=K))


@pytest.mark.parametrize("T", [75, 76, 77, 151, 152, 153, 305, 609])
def test_row_counts_around_the_forms(moe, T):
    """Row counts where the number of teams, of rows a team takes together and of CTAs changes."""
    for K in (64, 2880):
        d = rows(T, K, T, "token")
        check_forward(moe, d, "sigmoid", out8="ocp")
        check_backward(moe, *make_backward(d, "sigmoid", ck="ocp", seed=T))


@pytest.mark.parametrize("gate,ck,kw", [(None, None, {}), ("token", "ocp", {}), ("channel", "nosat", {}),
                                        ("token", None, dict(with_dy=False)), ("channel", None, dict(with_dh=False))])
def test_two_rows_a_team_and_an_odd_one_left(moe, gate, ck, kw):
    """The form for many long rows (T * K from 4.7 M on, rows past 2048 values), an odd number of them."""
    d = rows(2235, 2112, 31, gate, scaled=False)
    check_backward(moe, *make_backward(d, "sigmoid", ck=ck, seed=3, **kw))


def test_two_rows_a_team_keep_nan_in_their_row(moe):
    """A row of NaN beside a whole one, first and last: the other rows' gradients keep their bits."""
    d = rows(2235, 2112, 32, "token", scaled=False)
    call, _ = make_backward(d, "linear", seed=4)
    run = lambda: moe.sandwich_norm_backward(**{k: v if isinstance(v, str) else cuda(v) for k, v in call.items()})
    want = run()
    for t in (0, 1001, 2234):
        call["grad_y"][t, 7] = float("nan")
    got = run()
    keep = [t for t in range(2235) if t not in (0, 1001, 2234)]
    assert same(got.x[keep], want.x[keep]) and same(got.residual[keep], want.residual[keep])
    assert same(got.gate[keep], want.gate[keep]) and got.x[2234].isnan().all()


@pytest.mark.parametrize("e", [-60, -30, 30, 50])
def test_rows_far_from_one(moe, e):
    """Rows of magnitude 2^e without an eps: factors of 2^-e, whose squares are out of fp32's range at the ends."""
    for ck in (None, "nosat"):
        d = rows(9, 320, 4, "token", spread=0.1)
        d["x"] = (d["x"].float() * 2.0 ** e).bfloat16()
        d["residual"] = (d["residual"].float() * 2.0 ** e).bfloat16()
        d["gate"] = d["gate"] * 2.0 ** e          # the norm's output is of magnitude 1
        check_forward(moe, d, "linear", eps=0.0, out8="ocp", ck=ck)
        call, vals = make_backward(d, "linear", eps=0.0, ck=ck)
        r = check_backward(moe, call, vals)
        assert r.x.isfinite().all() and r.residual.isfinite().all()


def test_zero_gates_and_zero_scale(moe):
    for gate in ("channel", "token", "full"):
        d = rows(40, 320, 6, gate)
        d["gate"].zero_()
        d["residual_scale"].zero_()
        d["residual_scale"] += 0.5
        check_forward(moe, d, "linear", ck="ocp")
        r = check_backward(moe, *make_backward(d, "linear"))
        assert not r.x.any() and not r.post_gamma.any() and r.gate.any()
        d["residual_scale"].zero_()
        d["gate"].fill_(1.0)
        check_forward(moe, d, "linear")
        r = check_backward(moe, *make_backward(d, "linear"))
        assert not r.residual.any() and r.residual_scale.any()


def test_gates_far_out(moe):
    d = rows(16, 256, 8, "full", spread=0.1)
    d["gate"] = (d["gate"].float() * 40).bfloat16()
    d["gate"][0, :4] = torch.tensor([float("inf"), -float("inf"), 3e38, -3e38])
    check_forward(moe, d, "sigmoid")
    call, vals = make_backward(d, "sigmoid")
    r = check_backward(moe, call, vals)
    assert r.gate[0, :4].eq(0).all() and r.x.isfinite().all()


def test_column_sums_over_many_rows(moe):
    """Every row alike: the sums are T times a row's terms, to the roundings of T / 152 + 64 additions."""
    T, K = 100_003, 64
    d = rows(1, K, 9, None, scaled=True)
    call, vals = make_backward(d, "linear", seed=9)
    one = P.sandwich_norm_backward(**vals)
    for k in ("grad_h", "grad_y", "x", "h", "residual"):
        call[k] = call[k].expand(T, K).contiguous()
    call["rstd"] = call["rstd"].expand(2, T).contiguous()
    r = moe.sandwich_norm_backward(**{k: v if isinstance(v, str) else cuda(v) for k, v in call.items()})
    n = (T / 152 + 64) * 2.0 ** -24
    for name in ("pre_gamma", "post_gamma"):
        want = T * one[name]
        scale = np.abs(want).max()
        assert np.all(np.abs(f64(getattr(r, name)) - want) <= n * np.abs(want) + 2.0 ** -17 * scale)
    assert same(r.x[0], r.x[-1]) and same(r.x[0], r.x[T // 2])


def test_sandwich_norm_of_the_most_rows(moe):
    """2^31 - 1 rows (137 GB, in place, the stream beside itself): the row after a team's last one is past 2^31."""
    T, K = 2 ** 31 - 1, 32
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 150e9:
        pytest.skip("needs 150 GB of free device memory")
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").fill_(1.0)
    at = torch.tensor([0, 1215, 1216, 2 ** 30, 2 ** 31 - 3650, 2 ** 31 - 3649, T - 2, T - 1], device="cuda")
    vals = torch.arange(len(at), device="cuda").float()[:, None].expand(-1, K).bfloat16() + 2
    x[at] = vals
    r = moe.sandwich_norm(x, x, residual_out=x)
    torch.cuda.synchronize()
    assert r.y is None and r.h is x and torch.equal(x[at], 2 * vals)
    for a in (2, 2 ** 29 + 1, 2 ** 31 - 9000):
        assert (x[a:a + 1000] == 2).all()
    del x, r
    torch.cuda.empty_cache()


def test_routers_of_the_most_rows(moe):
    """2^31 - 1 rows of one expert (26 GB)."""
    T = 2 ** 31 - 1
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 50e9:
        pytest.skip("needs 50 GB of free device memory")
    x = torch.zeros(T, 1, device="cuda")
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    ids[-2] = -1
    off = torch.tensor([0, 2 ** 30 + 5, T], dtype=torch.int32, device="cuda")
    r = moe.router_balance(x, ids, "softmax", off)
    assert r.counts[:, 0].tolist() == [2 ** 30 + 5, T - 1 - (2 ** 30 + 5)]
    assert abs(float(r.stats[0]) - 1) <= 2.0 ** -20 and float(r.stats[1]) == 0 and float(r.stats[3]) == 2
    dw = torch.ones(T, 1, device="cuda")
    g = moe.router_backward(x, ids, dw, "sigmoid", renormalise=False, route_scale=4.0, grad_logits=dw)
    torch.cuda.synchronize()
    assert int((g == 1).sum()) == T - 1 and float(g[-2]) == 0
    del x, ids, dw, g
    torch.cuda.empty_cache()


def test_router_gradient_of_infinite_logits(moe):
    inf = float("inf")
    x = torch.tensor([[inf, 0.0, 1.0, -inf], [inf, inf, 0.0, 2.0], [0.0, inf, -inf, 1.0]])
    ids = torch.tensor([[0, 1], [0, 1], [3, 0]], dtype=torch.int32)
    dw = torch.tensor([[1.0, 2.0], [1.0, 3.0], [1.0, 5.0]])
    b = moe.router_balance(x.cuda(), ids.cuda(), "softmax")
    assert b.prob.isfinite().all() and b.stats[0].isfinite() and b.stats[1].isinf()
    assert torch.allclose(b.prob[0].cpu(), torch.tensor([0.5, 0.5, 0.0, 0.0]))
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            g = moe.router_backward(x.cuda(), ids.cuda(), dw.cuda(), scoring, renormalise=renorm,
                                    grad_losses=torch.tensor([1.0, 0.0]).cuda(), stats=b.stats, slope=b.slope)
            assert g.isfinite().all(), (scoring, renorm, g)
    # two infinite logits share the weight: q = 1/2 each, q (dw - mean) = -+1/2
    g = moe.router_backward(x[1:2].cuda(), ids[1:2].cuda(), dw[1:2].cuda(), "softmax")
    assert torch.allclose(g[0].cpu(), torch.tensor([-0.5, 0.5, 0.0, 0.0]))


def test_router_gradient_unaligned_rows(moe):
    """Logits that begin 4 bytes past a 16-byte boundary take the form without 16-byte loads: the same values."""
    T, E = 37, 64
    x, ids = torch.randn(T, E, generator=gen(2)), torch.randint(0, E, (T, 3), generator=gen(3), dtype=torch.int32)
    want = check_router_backward(moe, x, ids, "sigmoid", True)
    buf = torch.empty(T * E + 1, device="cuda")
    y = buf[1:].view(T, E)
    y.copy_(x)
    b = moe.router_balance(y, ids.cuda(), "sigmoid")
    c = moe.router_balance(x.cuda(), ids.cuda(), "sigmoid")
    assert torch.equal(b.counts, c.counts)
    # the lanes hold other experts, so the sums over a row run in another order: 40 roundings at most
    assert torch.allclose(b.prob, c.prob, rtol=2.0 ** -17, atol=0)
    got = moe.router_backward(y, ids.cuda(), torch.randn(T, 3, generator=gen(0)).cuda(), "sigmoid", renormalise=True,
                              route_scale=1.7, grad_losses=torch.tensor([0.7, 0.05]).cuda(), stats=c.stats,
                              slope=c.slope)
    assert torch.allclose(got, want, rtol=2.0 ** -14, atol=1e-6)


def test_many_sequences_of_one_token_and_many_empty_ones(moe):
    T, S = 3000, 1 << 17
    x = torch.randn(T, 16, generator=gen(4))
    ids = torch.randint(0, 16, (T, 2), generator=gen(5), dtype=torch.int32)
    off = torch.sort(torch.randint(0, T + 1, (S + 1,), generator=gen(6))).values.int()
    r = moe.router_balance(x.cuda(), ids.cuda(), "softmax", off.cuda())
    o = P.router_balance(x.numpy(), ids.numpy(), "softmax", off.tolist())
    assert np.array_equal(r.counts.cpu().numpy(), o["counts"])
    assert abs(float(r.stats[0]) - o["stats"][0]) <= 2.0 ** -16 * o["stats"][0]
    assert float(r.stats[2]) == o["stats"][2] and float(r.stats[3]) == o["stats"][3]


def test_parameters_and_views_are_taken(moe):
    d = rows(8, 128, 11, "channel")
    c = {k: cuda(v) for k, v in d.items()}
    want = moe.sandwich_norm(**c)
    p = {k: torch.nn.Parameter(v) for k, v in c.items()}
    got = moe.sandwich_norm(**p)
    assert same(got.y, want.y) and not got.y.requires_grad
    wide = torch.stack((c["x"], c["x"]))          # rows of a larger buffer, at an offset
    assert same(moe.sandwich_norm(**{**c, "x": wide[1]}).y, want.y)
    with pytest.raises(ValueError):
        moe.sandwich_norm(**{**c, "x": c["x"].cpu()})
    with pytest.raises(ValueError):
        moe.sandwich_norm(**{**c, "pre_gamma": c["pre_gamma"].cpu()})


FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import test_block_gradients_gpu as B
from mxfp4_mixture_experts_gb300 import moe
K = {K}
f, _ = B.calls(moe, T=40, K=K)[{op!r}] if {op!r} != "sandwich_norm_backward" else (None, 0)
if f is None:
    call, _ = B.make_backward(B.rows(40, K, 21, "full"), "sigmoid", seed=1)
    call = {{n: v if isinstance(v, str) else B.cuda(v) for n, v in call.items()}}
    f = lambda **kw: moe.sandwich_norm_backward(**call, **kw)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = f()
g.replay()
torch.cuda.synchronize()
assert B.same(B.copies(out), B.copies(f()))
print("same")
"""


@pytest.mark.parametrize("op,K", [("sandwich_norm", 640), ("sandwich_norm_backward", 640), ("sandwich_norm_backward", 8224),
                                  ("router_backward", 640), ("combine_backward", 640)])
def test_first_call_of_a_process_inside_a_capture(moe, op, K):
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=os.path.dirname(tests), tests=tests, op=op, K=K)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
