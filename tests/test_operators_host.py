"""The operators around the layer, without a GPU: host refusals of the C ABI, and
pins of their float64 oracle against hand cases and second formulations."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

from oracle import mxfp4_moe_oracle as O
from oracle import operators_oracle as P

VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    from mxfp4_mixture_experts_gb300 import moe
    return moe


def norm(m, **kw):
    a = dict(x=VP(0x10000), res=VP(0x20000), gamma=VP(0x30000), T=4, K=64, eps=1e-5, rule=0,
             res_out=VP(0x40000), out=VP(0x50000), q=VP(0x60000), s=VP(0x70000), stream=None)
    a.update(kw)
    return m.lib().mxfp4_moe_add_rmsnorm(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(K=48), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=16416), "SHAPE"), (dict(T=-1), "SHAPE"),
    (dict(eps=-1.0), "ARG"), (dict(eps=float("nan")), "ARG"), (dict(eps=float("inf")), "ARG"),
    (dict(rule=2), "ARG"), (dict(s=None), "ARG"), (dict(q=None), "ARG"), (dict(x=None), "ARG"),
    (dict(gamma=None), "ARG"), (dict(out=None, q=None, s=None, res_out=None), "ARG"),
    (dict(x=VP(0x10008)), "ALIGN"), (dict(res=VP(0x20002)), "ALIGN"), (dict(q=VP(0x60008)), "ALIGN"),
    (dict(out=VP(0x50008)), "ALIGN"), (dict(T=0, x=None), "OK"),
])
def test_add_rmsnorm_refusals(m, kw, code):
    want = m.OK if code == "OK" else getattr(m, "ERR_" + code)
    assert norm(m, **kw) == want


def router(m, **kw):
    a = dict(logits=VP(0x10000), bias=VP(0x20000), T=4, E=64, k=4, scoring=1, n_group=8,
             topk_group=4, group_top=2, renorm=1, scale=1.0, ids=VP(0x30000), w=VP(0x40000),
             stream=None)
    a.update(kw)
    return m.lib().mxfp4_moe_router_scored(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(E=1025, n_group=1, topk_group=1), "SHAPE"), (dict(E=0), "SHAPE"), (dict(k=33), "SHAPE"),
    (dict(k=0), "SHAPE"), (dict(n_group=7), "SHAPE"), (dict(topk_group=9), "SHAPE"),
    (dict(topk_group=1, k=9), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(scoring=2), "ARG"),
    (dict(group_top=3), "ARG"), (dict(renorm=2), "ARG"), (dict(scale=float("nan")), "ARG"),
    (dict(scale=float("inf")), "ARG"), (dict(logits=None), "ARG"), (dict(ids=None), "ARG"),
    (dict(bias=VP(0x20002)), "ALIGN"), (dict(w=VP(0x40001)), "ALIGN"), (dict(T=0, logits=None), "OK"),
])
def test_router_scored_refusals(m, kw, code):
    want = m.OK if code == "OK" else getattr(m, "ERR_" + code)
    assert router(m, **kw) == want


def lin(m, **kw):
    a = dict(x=VP(0x10000), xs=None, w=VP(0x20000), s=VP(0x30000), T=4, K=128, N=64,
             ids=VP(0x40000), a=VP(0x50000), b=VP(0x60000), scale=VP(0x70000), L=3, rank=16,
             out=VP(0x80000), status=None, ws=VP(0x100000), ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return m.lib().mxfp4_moe_linear(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(K=96), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=16448), "SHAPE"), (dict(N=12), "SHAPE"),
    (dict(N=0), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(T=(1 << 20) + 1), "SHAPE"),
    (dict(rank=12), "SHAPE"), (dict(rank=0), "SHAPE"), (dict(rank=264), "SHAPE"),
    (dict(L=0), "SHAPE"), (dict(L=1025), "SHAPE"), (dict(x=None), "ARG"), (dict(w=None), "ARG"),
    (dict(s=None), "ARG"), (dict(out=None), "ARG"), (dict(a=None), "ARG"), (dict(b=None), "ARG"),
    (dict(x=VP(0x10010)), "ALIGN"), (dict(xs=VP(0x10008)), "ALIGN"), (dict(w=VP(0x20004)), "ALIGN"),
    (dict(ids=VP(0x40002)), "ALIGN"), (dict(a=VP(0x50010)), "ALIGN"), (dict(out=VP(0x80008)), "ALIGN"),
    (dict(ws=VP(0x100080)), "ALIGN"), (dict(ws=None), "WORKSPACE"), (dict(ws_bytes=0), "WORKSPACE"),
    (dict(T=0, x=None, ids=None), "OK"),
])
def test_linear_refusals(m, kw, code):
    want = m.OK if code == "OK" else getattr(m, "ERR_" + code)
    assert lin(m, **kw) == want


def test_linear_workspace_size(m):
    f = m.linear_workspace_size
    assert f(4, 96, 64, 16) == 0 and f(4, 128, 64, 12) == 0 and f(-1, 128, 64) == 0
    assert f(4, 128, 64, 16) > 0
    assert f(400, 128, 64, 16) > f(4, 128, 64, 16)


def test_binding_refuses_wrong_tensors(m):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m.add_rmsnorm(x, torch.ones(64, dtype=torch.bfloat16))          # not on a GPU
    with pytest.raises(TypeError):
        m.add_rmsnorm(x.float(), torch.ones(64, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        m.router_scored(x, 2)
    with pytest.raises(TypeError):
        m.linear(x.float(), None, None)
    with pytest.raises(TypeError):
        m.linear(x, None, None, x_scale=torch.zeros(2, 2, dtype=torch.uint8))   # bf16 with scales


# ------------------------------------------------------------------ oracle pins
def test_e4m3_table_matches_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes.copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(P.e4m3_value(codes), want, equal_nan=True)


def test_round_e4m3_is_nearest_even_over_all_neighbours():
    v = np.sort(P.e4m3_value(np.arange(127, dtype=np.uint8)))
    lo, hi = v[:-1], v[1:]
    mid = (lo + hi) / 2
    assert np.array_equal(P.round_e4m3(np.nextafter(mid, 0)), lo)
    assert np.array_equal(P.round_e4m3(np.nextafter(mid, 1e9)), hi)
    even = np.where(np.arange(126) % 2 == 0, lo, hi)      # the code with an even last bit
    assert np.array_equal(P.round_e4m3(mid), even)
    assert P.round_e4m3(1e9) == 448 and P.round_e4m3(-465) == -448


def test_mx8_exponent_by_hand():
    assert P.mx8_exponent(256.0, "ocp") == 0 and P.mx8_exponent(511.9, "ocp") == 0
    assert P.mx8_exponent(448.0, "nosat") == 0 and P.mx8_exponent(448.1, "nosat") == 1
    assert P.mx8_exponent(512.0, "nosat") == 1 and P.mx8_exponent(0.0, "ocp") == -127
    assert P.mx8_exponent(1.0, "ocp") == -8 and P.mx8_exponent(2.0 ** -140, "ocp") == -127


def test_add_rmsnorm_closed_form():
    x = np.full((1, 64), 3.0)
    bits = O.float_to_bf16_bits(x)
    gamma = O.float_to_bf16_bits(np.arange(64) / 32.0)
    h, y = P.add_rmsnorm(bits, gamma, 0.0)
    assert np.allclose(y, np.arange(64) / 32.0, rtol=1e-15)
    h, y = P.add_rmsnorm(bits, gamma, 0.0, O.float_to_bf16_bits(-x))
    assert np.all(h == 0) and np.all(np.isnan(y))
    _, y = P.add_rmsnorm(bits, gamma, 7.0)          # 3 / sqrt(9 + 7)
    assert np.allclose(y, 0.75 * np.arange(64) / 32.0, rtol=1e-15)


def test_router_bias_on_scores_orders_unlike_bias_on_logits():
    # sigmoid(4) = .982, sigmoid(0) = .5: a bias of .6 lifts the second on scores, not on logits
    ids, w, _ = P.router_scored([[4.0, 0.0]], 1, "sigmoid", [0.0, 0.6])
    assert ids[0, 0] == 1 and w[0, 0] == 1.0
    ids, w, _ = P.router_scored([[4.0, 0.0]], 1, "sigmoid", [0.0, 0.6], renormalise=False, route_scale=2.0)
    assert abs(w[0, 0] - 1.0) < 1e-15                # 2 * sigmoid(0)


def test_router_group_by_best_two_by_hand():
    # group sums of two: .9 + .1 against .6 + .55; by the largest alone group 0 wins
    p = np.array([[0.9, 0.1, 0.6, 0.55]])
    x = np.log(p / (1 - p))
    assert list(P.router_scored(x, 2, "sigmoid", None, 2, 1)[0][0]) == [2, 3]
    assert list(P.router_scored(x, 2, "sigmoid", None, 2, 1, group_top=1)[0][0]) == [0, 1]


def test_router_masked_experts_and_empty_rows():
    inf, nan = np.inf, np.nan
    ids, w, _ = P.router_scored([[-inf, 1.0, nan, -inf], [-inf] * 4], 2, "softmax")
    assert list(ids[0]) == [1, -1] and list(w[0]) == [1.0, 0.0]
    assert list(ids[1]) == [-1, -1] and list(w[1]) == [0.0, 0.0]


def test_router_against_enumeration():
    rng = np.random.default_rng(3)
    for _ in range(20):
        x, b = rng.normal(size=(1, 6)), rng.normal(size=6) * 0.2
        ids, w, _ = P.router_scored(x, 3, "softmax", b, renormalise=False)
        s = np.exp(x[0]) / np.exp(x[0]).sum()
        best = max(itertools.permutations(range(6), 3),
                   key=lambda p: tuple(s[e] + b[e] for e in p))
        assert list(ids[0]) == list(best)
        assert np.allclose(w[0], s[list(best)], rtol=1e-14)


def test_linear_adapter_closed_form():
    """Zero weights leave the adapter alone; a rank-8 identity picks the first inputs."""
    K, N, r = 64, 16, 8
    x = np.arange(2 * K, dtype=np.float64).reshape(2, K)
    w, s = np.zeros((N, K // 2), np.uint8), np.full((N, K // 32), 127, np.uint8)
    a = np.zeros((2, r, K)); a[1, np.arange(r), np.arange(r)] = 1
    b = np.zeros((2, N, r)); b[1, np.arange(r), np.arange(r)] = 1
    y, _, _ = P.linear(x, w, s, [1, 5], O.float_to_bf16_bits(a), O.float_to_bf16_bits(b), [1.0, 3.0])
    assert np.array_equal(y[0, :r], 3 * x[0, :r]) and not y[0, r:].any() and not y[1].any()
    w[:] = 0x22                                       # every code 2: the value 1
    y, _, _ = P.linear(x, w, s, [0, -1], O.float_to_bf16_bits(a), O.float_to_bf16_bits(b))
    assert np.array_equal(y, np.repeat(x.sum(1, keepdims=True), N, 1))
