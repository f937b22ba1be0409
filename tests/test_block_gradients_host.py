"""The operators that train what stands around the experts, without a GPU: host refusals of the C ABI
and of the binding, and pins of their float64 oracle against differences, hand cases and torch."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import operators_oracle as P

VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    from mxfp4_mixture_experts_gb300 import moe
    return moe


def check(m, rc, code):
    assert rc == (m.OK if code == "OK" else getattr(m, "ERR_" + code))


def sandwich(m, **kw):
    a = dict(x=VP(0x10000), res=VP(0x20000), post=VP(0x30000), pre=VP(0x40000), gate=VP(0x50000), kind=1, act=0,
             scale=VP(0x60000), T=4, K=64, eps=1e-5, rule=0, ck=0, h=VP(0x70000), out=VP(0x80000), q=VP(0x90000),
             qs=VP(0xa0000), x8=VP(0xb0000), xs=VP(0xc0000), h8=VP(0xd0000), hs=VP(0xe0000), rstd=VP(0xf0000),
             stream=None)
    a.update(kw)
    return m.lib().mxfp4_moe_sandwich_norm(*a.values())


NONE = dict(h=None, out=None, q=None, qs=None, x8=None, xs=None, h8=None, hs=None, rstd=None)


@pytest.mark.parametrize("kw,code", [
    (dict(K=48), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=16416), "SHAPE"), (dict(T=-1), "SHAPE"),
    (dict(eps=-1.0), "ARG"), (dict(eps=float("nan")), "ARG"), (dict(eps=float("inf")), "ARG"),
    (dict(rule=2), "ARG"), (dict(ck=-1), "ARG"), (dict(kind=4), "ARG"), (dict(kind=0), "ARG"),
    (dict(gate=None), "ARG"), (dict(act=2), "ARG"), (dict(x=None), "ARG"), (dict(res=None), "ARG"),
    (dict(q=None), "ARG"), (dict(xs=None), "ARG"), (dict(h8=None), "ARG"), (dict(pre=None), "ARG"),
    (dict(pre=None, out=None), "ARG"), (NONE, "ARG"), (dict(x=VP(0x10008)), "ALIGN"),
    (dict(res=VP(0x20002)), "ALIGN"), (dict(post=VP(0x30008)), "ALIGN"), (dict(gate=VP(0x50004)), "ALIGN"),
    (dict(gate=VP(0x50002), kind=2), "ALIGN"), (dict(scale=VP(0x60002)), "ALIGN"),
    (dict(h8=VP(0xd0008)), "ALIGN"), (dict(rstd=VP(0xf0001)), "ALIGN"), (dict(T=0, x=None), "OK"),
])
def test_sandwich_norm_refusals(m, kw, code):
    check(m, sandwich(m, **kw), code)


def sandwich_bwd(m, **kw):
    a = dict(dh=VP(0x10000), dy=VP(0x20000), x=VP(0x30000), xs=None, h=VP(0x40000), hs=None, rstd=VP(0x50000),
             post=VP(0x60000), pre=VP(0x70000), gate=VP(0x80000), kind=3, act=1, res=VP(0x90000),
             scale=VP(0xa0000), T=4, K=64, dx=VP(0xb0000), dres=VP(0xc0000), dpost=VP(0xd0000),
             dpre=VP(0xe0000), dgate=VP(0xf0000), dscale=VP(0x100000), ws=VP(0x200000), n=1 << 40, stream=None)
    a.update(kw)
    return m.lib().mxfp4_moe_sandwich_norm_backward(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(K=48), "SHAPE"), (dict(K=16416), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(kind=-1), "ARG"),
    (dict(act=2), "ARG"), (dict(gate=None), "ARG"), (dict(kind=0), "ARG"), (dict(kind=0, gate=None), "ARG"),
    (dict(post=None), "ARG"), (dict(pre=None), "ARG"), (dict(pre=None, dpre=None), "ARG"),
    (dict(scale=None), "ARG"), (dict(res=None), "ARG"), (dict(dh=None, dy=None), "ARG"), (dict(x=None), "ARG"),
    (dict(h=None), "ARG"), (dict(rstd=None), "ARG"),
    (dict(dx=None, dres=None, dpost=None, dpre=None, dgate=None, dscale=None), "ARG"),
    (dict(dh=VP(0x10008)), "ALIGN"), (dict(x=VP(0x30004)), "ALIGN"), (dict(dgate=VP(0xf0004)), "ALIGN"),
    (dict(dpre=VP(0xe0004)), "ALIGN"), (dict(ws=VP(0x200080)), "ALIGN"), (dict(ws=None), "WORKSPACE"),
    (dict(n=4), "WORKSPACE"),
])
def test_sandwich_norm_backward_refusals(m, kw, code):
    check(m, sandwich_bwd(m, **kw), code)


def balance(m, **kw):
    a = dict(x=VP(0x10000), ids=VP(0x20000), T=4, E=64, k=4, scoring=1, off=VP(0x30000), S=3, stats=VP(0x40000),
             counts=VP(0x50000), prob=VP(0x60000), slope=VP(0x70000), ws=VP(0x80000), n=1 << 40, stream=None)
    a.update(kw)
    return m.lib().mxfp4_moe_router_balance(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(E=1025), "SHAPE"), (dict(E=0), "SHAPE"), (dict(k=0), "SHAPE"), (dict(k=33), "SHAPE"),
    (dict(E=3), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(T=2 ** 29), "SHAPE"), (dict(S=0), "SHAPE"),
    (dict(S=2 ** 20 + 1), "SHAPE"), (dict(scoring=2), "ARG"), (dict(off=None), "ARG"), (dict(x=None), "ARG"),
    (dict(ids=None), "ARG"), (dict(stats=None), "ARG"), (dict(counts=None), "ARG"), (dict(slope=None), "ARG"),
    (dict(x=VP(0x10002)), "ALIGN"), (dict(off=VP(0x30001)), "ALIGN"), (dict(prob=VP(0x60002)), "ALIGN"),
    (dict(ws=VP(0x80010)), "ALIGN"), (dict(ws=None), "WORKSPACE"), (dict(n=64), "WORKSPACE"),
])
def test_router_balance_refusals(m, kw, code):
    check(m, balance(m, **kw), code)


def router_bwd(m, **kw):
    a = dict(x=VP(0x10000), ids=VP(0x20000), dw=VP(0x30000), T=4, E=64, k=4, scoring=1, renorm=1, scale=1.0,
             dloss=VP(0x40000), stats=VP(0x50000), slope=VP(0x60000), off=VP(0x70000), S=3, dx=VP(0x80000),
             stream=None)
    a.update(kw)
    return m.lib().mxfp4_moe_router_backward(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(E=1025), "SHAPE"), (dict(k=33), "SHAPE"), (dict(E=3), "SHAPE"), (dict(T=-1), "SHAPE"),
    (dict(T=2 ** 29), "SHAPE"), (dict(S=0), "SHAPE"), (dict(scoring=-1), "ARG"), (dict(renorm=2), "ARG"),
    (dict(scale=float("inf")), "ARG"), (dict(scale=float("nan")), "ARG"), (dict(off=None), "ARG"),
    (dict(x=None), "ARG"), (dict(ids=None), "ARG"), (dict(dx=None), "ARG"), (dict(dw=None, dloss=None), "ARG"),
    (dict(stats=None), "ARG"), (dict(slope=None), "ARG"), (dict(dw=VP(0x30002)), "ALIGN"),
    (dict(slope=VP(0x60001)), "ALIGN"), (dict(T=0, x=None), "OK"),
])
def test_router_backward_refusals(m, kw, code):
    check(m, router_bwd(m, **kw), code)


def combine(m, **kw):
    a = dict(dy=VP(0x10000), o=VP(0x20000), ids=VP(0x30000), w=VP(0x40000), T=4, K=64, k=4, base=0, E=8,
             dw=VP(0x50000), do=VP(0x60000), stream=None)
    a.update(kw)
    return m.lib().mxfp4_moe_combine_backward(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(K=40), "SHAPE"), (dict(K=16416), "SHAPE"), (dict(k=0), "SHAPE"), (dict(k=33), "SHAPE"),
    (dict(T=-1), "SHAPE"), (dict(T=2 ** 29), "SHAPE"), (dict(E=-1), "SHAPE"), (dict(base=-1), "ARG"),
    (dict(dy=None), "ARG"), (dict(o=None), "ARG"), (dict(dw=None), "ARG"), (dict(w=None), "ARG"),
    (dict(o=VP(0x20008)), "ALIGN"), (dict(ids=VP(0x30002)), "ALIGN"), (dict(do=VP(0x60004)), "ALIGN"),
    (dict(T=0, dy=None), "OK"),
])
def test_combine_backward_refusals(m, kw, code):
    check(m, combine(m, **kw), code)


def test_workspace_sizes(m):
    f, b = m.sandwich_norm_backward_workspace_size, m.router_balance_workspace_size
    assert f(4, 48) == 0 and f(-1, 64) == 0 and 0 < f(4, 64) < f(400, 64) <= f(10 ** 6, 64)
    assert b(4, 1025) == 0 and b(4, 64, 0) == 0 and 0 < b(4, 64) < b(4, 64, 9) < b(4000, 64, 9)
    assert b(0, 8) > 0


def test_binding_refuses_wrong_tensors(m):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m.sandwich_norm(bf(2, 64), bf(2, 64))                              # not on a GPU
    with pytest.raises(TypeError):
        m.sandwich_norm(bf(2, 64).float(), bf(2, 64))
    with pytest.raises(ValueError):
        m.sandwich_norm_backward(None, None, bf(2, 64), None, None)
    with pytest.raises(TypeError):
        m.sandwich_norm_backward(bf(2, 64), None, bf(2, 64), None, None, x_scale=torch.zeros(2, 2).byte())
    with pytest.raises(TypeError):
        m.router_balance(bf(2, 8), torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(TypeError):
        m.router_backward(bf(2, 8), torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(TypeError):
        m.combine_backward(bf(2, 64).float(), bf(4, 64))


# ------------------------------------------------------------------ oracle pins
def differences(f, x, eps=1e-6):
    """Central differences of the scalar f at every entry of x."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


@pytest.mark.parametrize("act", ["linear", "sigmoid"])
@pytest.mark.parametrize("gshape", [None, (1, 8), (3, 1), (3, 8)])
@pytest.mark.parametrize("post", [True, False])
def test_sandwich_gradient_against_differences(gshape, act, post):
    """Central differences of float64: an error of eps^2 f''' / 6 and 2^-52 |f| / eps, below 1e-7 here."""
    rng = np.random.default_rng(5)
    v = dict(x=rng.normal(size=(3, 8)), residual=rng.normal(size=(3, 8)) * 2, pre_gamma=1 + 0.3 * rng.normal(size=8),
             scale=np.array(0.7))
    if post:
        v["post_gamma"] = 0.5 + 0.3 * rng.normal(size=8)
    if gshape:
        v["gate"] = rng.normal(size=gshape)
    dh, dy = rng.normal(size=(3, 8)), rng.normal(size=(3, 8))

    def loss(**kw):
        r = P.sandwich_norm(**{**v, **kw}, act=act, eps=0.3)
        return float(np.sum(dh * r["h"]) + np.sum(dy * r["y"]))

    r = P.sandwich_norm(**v, act=act, eps=0.3)
    g = P.sandwich_norm_backward(dh, dy, v["x"], r["h"], r["r1"], r["r2"], v.get("post_gamma"), v["pre_gamma"],
                                 v.get("gate"), act, v["residual"], v["scale"])
    names = dict(x="x", residual="residual", pre_gamma="pre_gamma", residual_scale="scale")
    if post:
        names["post_gamma"] = "post_gamma"
    for got, name in names.items():
        want = differences(lambda a: loss(**{name: a}), v[name])
        assert np.allclose(g[got], want, rtol=0, atol=1e-7 * (1 + np.abs(want).max())), got
    if gshape:
        full = g["gate"]
        for ax in (0, 1):
            if gshape[ax] == 1:
                full = full.sum(ax, keepdims=True)
        assert np.allclose(full, differences(lambda a: loss(gate=a), v["gate"]), rtol=0, atol=1e-6)


def test_sandwich_closed_forms():
    x, res = np.full((1, 4), 3.0), np.full((1, 4), 2.0)
    r = P.sandwich_norm(x, res, np.ones(4), np.ones(4), np.full((1, 1), 2.0), eps=0.0)
    assert np.allclose(r["h"], 4.0) and np.allclose(r["y"], 1.0) and np.allclose(r["r1"], 1 / 3)
    # a gradient along h leaves no trace through a norm without eps
    g = P.sandwich_norm_backward(None, r["h"], x, r["h"], r["r1"], r["r2"], np.ones(4), np.ones(4), np.full((1, 1), 2.0))
    assert np.allclose(g["residual"], 0, atol=1e-15) and np.allclose(g["x"], 0, atol=1e-15)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_router_gradient_against_differences(scoring, renormalise):
    rng = np.random.default_rng(7)
    x = rng.normal(size=(7, 5))
    ids = np.array([[0, 1], [3, 3], [4, -1], [-1, -1], [9, 2], [1, 0], [2, 4]])
    off = np.array([0, 3, 3, 6])
    dw, dl = rng.normal(size=(7, 2)), np.array([0.6, 0.3])

    def loss(z):
        return float(np.sum(dw * P.router_weights(z, ids, scoring, renormalise, 1.7))
                     + dl @ P.router_balance(z, ids, scoring, off)["stats"][:2])

    g, _ = P.router_backward(x, ids, dw, scoring, renormalise, 1.7, dl, P.router_balance(x, ids, scoring, off))
    assert np.allclose(g, differences(loss, x), rtol=0, atol=1e-7)


def test_balance_closed_forms():
    # an even routing of even scores has loss 1, one expert for all E
    x = np.zeros((8, 4))
    even = P.router_balance(x, np.arange(8)[:, None] % 4, "softmax")
    assert abs(even["stats"][0] - 1) < 1e-15 and abs(even["stats"][1] - np.log(4) ** 2) < 1e-15
    x[:, 2] = 50.0
    one = P.router_balance(x, np.full((8, 1), 2), "softmax")
    assert abs(one["stats"][0] - 4) < 1e-12 and list(one["counts"][0]) == [0, 0, 8, 0]
    none = P.router_balance(x, np.full((8, 1), -1), "softmax", [0, 4, 8])
    assert not none["stats"].any() and not none["slope"].any()


def test_combine_against_torch():
    g = torch.Generator().manual_seed(3)
    w = torch.randn(3, 2, generator=g, dtype=torch.float64, requires_grad=True)
    o = torch.randn(3, 2, 8, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(3, 8, generator=g, dtype=torch.float64)
    ((w[:, :, None] * o).sum(1) * dy).sum().backward()
    dw, _, do = P.combine_backward(dy.numpy(), o.detach().numpy(), None, w.detach().numpy())
    assert np.allclose(dw, w.grad.numpy(), rtol=1e-14) and np.allclose(do, o.grad.numpy(), rtol=1e-14)
    dw, _, do = P.combine_backward(dy.numpy(), o.detach().numpy(), [[0, 5], [-1, 4], [3, 2]], w.detach().numpy(), 2, 3)
    assert (dw != 0).tolist() == [[False, False], [False, True], [True, True]]
