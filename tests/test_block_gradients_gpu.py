"""The operators that train what stands around the experts, against their float64 oracle.

Tolerances, from the operators' own roundings (u = 2^-24; sums of K terms take at most 32 serial additions a
thread and 15 in trees, so an error of at most 47 u, below S = 2^-18, times the sum of magnitudes):
* r1, r2: half of S, the root 2 u: below R = 2^-18 relative;
* n = x r1 gamma: R and two roundings; a gate's sigmoid (expf 2 ulp, an addition, a reciprocal): 2^-21; h: one
  product, one fused addition: below 2^-17 of |g n| + |scale res| in all; bf16 adds 2^-8 of the value;
* y: h's error, r2's (R and the row's relative error of h), 2^-8 in bf16, half a step in MXFP8;
* gradient: as derived beside ``sandwich_tolerances``;
* p: expf 2 ulp, sums of at most 32 + 5 non-negative terms, a quotient: below 2^-18 relative; logarithm and its
  addition: 2^-18 + 2^-22 |lse| absolute;
* the router's gradient: a handful of such products, sums of at most 37 terms: 2^-16 of the terms' magnitudes."""
import numpy as np
import pytest
import torch

from oracle import mxfp4_moe_oracle as O
from oracle import operators_oracle as P

pytestmark = pytest.mark.gpu
S = R = 2.0 ** -18
BF = 2.0 ** -8
TINY = 2.0 ** -126


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    from mxfp4_mixture_experts_gb300 import moe
    return moe


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def cuda(t):
    return None if t is None else t.cuda()


def same(a, b):
    """Bit for bit, tuple by tuple."""
    if a is None or isinstance(a, torch.Tensor):
        return (a is None and b is None) or torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    return len(a) == len(b) and all(same(x, y) for x, y in zip(a, b))


def rows(T, K, seed, gate=None, post=True, pre=True, scaled=True, spread=1.0):
    g = gen(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    d = dict(x=(rn(T, K) * torch.exp(spread * rn(T, 1))).bfloat16(), residual=(3 * rn(T, K)).bfloat16(),
             post_gamma=(0.5 + 0.2 * rn(K)).bfloat16() if post else None,
             pre_gamma=(1 + 0.3 * rn(K)).bfloat16() if pre else None, gate=None,
             residual_scale=0.5 + torch.rand(1, generator=g) if scaled else None)
    if gate == "channel":
        d["gate"] = rn(1, K).bfloat16()
    elif gate == "token":
        d["gate"] = rn(T, 1)
    elif gate == "full":
        d["gate"] = rn(T, K).bfloat16()
    return d


def oracle_forward(d, act, eps):
    a = d["residual_scale"]
    return P.sandwich_norm(f64(d["x"]), f64(d["residual"]), f64(d["post_gamma"]), f64(d["pre_gamma"]), f64(d["gate"]),
                           act, None if a is None else float(a[0]), eps)


def check_mx8(q, s, y, dy, rule):
    """E4M3 values q and scale bytes s of y, itself known to within dy: the exponent of the block's largest
    magnitude or of one within dy of it, each value within half a step and dy."""
    T, K = y.shape
    block = lambda v: v.reshape(T, K // 32, 32)
    q, s = f64(q), s.cpu().numpy().astype(np.int64)
    a = np.abs(block(y))
    lo, hi = np.maximum(a - block(dy), 0).max(-1), (a + block(dy)).max(-1)
    X = np.vectorize(lambda v: P.mx8_exponent(float(v), rule))
    assert np.all((s >= X(lo) + 127) & (s <= X(hi) + 127))
    f = np.exp2(np.repeat(s, 32, 1) - 127.0)
    v, dv = np.abs(y) / f, dy / f
    _, e = np.frexp(np.minimum(v + dv, 448.0))
    half = np.exp2(np.maximum(e - 1, -6) - 4.0)
    assert np.all(np.abs(q - np.sign(y) * np.minimum(v, 448.0)) <= half + dv)


def check_forward(moe, d, act="linear", eps=1e-5, out8=None, ck=None, **kw):
    c = {k: cuda(v) for k, v in d.items()}
    if "in_place" in kw:
        kw["residual_out"] = c[kw.pop("in_place")]
    r = moe.sandwich_norm(**c, gate_act=act, eps=eps, out8=out8, checkpoint8=ck, rstd=True, **kw)
    torch.cuda.synchronize()
    o = oracle_forward(d, act, eps)
    a = 1.0 if d["residual_scale"] is None else float(d["residual_scale"])
    g = P.gate_values(f64(d["gate"]), act)[0]
    dh = 2.0 ** -17 * (np.abs(g * o["n"]) + np.abs(a * f64(d["residual"]))) + TINY
    h = o["h"]
    assert np.all(np.abs(f64(r.h) - h) <= dh + BF * np.abs(h))
    rel = np.linalg.norm(dh, axis=1) / (np.linalg.norm(h, axis=1) + TINY) + R
    rs = f64(r.rstd)
    assert np.all(np.abs(rs[0] - o["r1"]) <= R * o["r1"])
    if d["pre_gamma"] is not None:
        assert np.all(np.abs(rs[1] - o["r2"]) <= rel * o["r2"])
        y = o["y"]
        dy = np.abs(o["r2"][:, None] * f64(d["pre_gamma"])) * dh + rel[:, None] * np.abs(y) + TINY
        if kw.get("bf16", True):
            assert np.all(np.abs(f64(r.y) - y) <= dy + BF * np.abs(y))
        if out8:
            check_mx8(r.q, r.q_scale, y, dy, out8)
    else:
        assert r.y is None and np.all(rs[1] == 1)
    if ck:
        check_mx8(r.x8, r.x8_scale, f64(d["x"]), np.zeros(h.shape), ck)
        check_mx8(r.h8, r.h8_scale, h, dh, ck)
    return r


SHAPES = [(1, 32), (1, 2880), (3, 64), (2, 7168), (5, 8160), (2, 8192), (1, 16384), (33, 1056), (700, 96), (5, 4128),
          (350, 512), (3, 8224), (190, 12320)]


@pytest.mark.parametrize("T,K", SHAPES)
@pytest.mark.parametrize("gate,act", [(None, "linear"), ("channel", "linear"), ("token", "sigmoid"), ("full", "sigmoid"),
                                      ("full", "linear"), ("channel", "sigmoid"), ("token", "linear")])
def test_sandwich_matches_oracle(moe, T, K, gate, act):
    check_forward(moe, rows(T, K, T + K, gate), act, out8="ocp", ck="nosat")
    check_forward(moe, rows(T, K, T + K + 1, gate, scaled=False), act, 1e-6)


@pytest.mark.parametrize("post,pre", [(False, True), (True, False), (False, False)])
def test_sandwich_without_a_norm(moe, post, pre):
    for gate in (None, "channel", "token", "full"):
        check_forward(moe, rows(40, 1056, 7, gate, post, pre), ck="ocp", out8="nosat" if pre else None)


@pytest.mark.parametrize("which", ["x", "residual"])
def test_sandwich_in_place(moe, which):
    for K in (256, 2880):
        check_forward(moe, rows(700, K, 8, "full"), out8="ocp", in_place=which)


def test_sandwich_outputs_alone(moe):
    d = {k: cuda(v) for k, v in rows(9, 320, 9, "channel").items()}
    a = moe.sandwich_norm(**d, out8="ocp", checkpoint8="ocp", rstd=True)
    b = moe.sandwich_norm(**d, out8="ocp", bf16=False)
    assert b.y is None and b.x8 is None and b.rstd is None and same(a.q, b.q) and same(a.q_scale, b.q_scale)
    assert same(a.h, moe.sandwich_norm(**{**d, "pre_gamma": None}).h)
    e = moe.sandwich_norm(d["x"][:0], d["residual"][:0], d["post_gamma"], d["pre_gamma"], out8="ocp", rstd=True)
    assert e.y.shape == (0, 320) and e.q_scale.shape == (0, 10) and e.rstd.shape == (2, 0)


def test_sandwich_nonfinite_and_zero_rows_stay_in_their_rows(moe):
    d = rows(6, 96, 10, "full")
    d["x"][0] = 0
    d["residual"][0] = 0
    d["x"][1, 40] = float("nan")
    d["x"][2, 3] = float("inf")
    d["residual"][3, 5] = float("inf")
    d["gate"][4, 7] = float("nan")
    r = moe.sandwich_norm(**{k: cuda(v) for k, v in d.items()}, out8="ocp", checkpoint8="ocp", rstd=True)
    torch.cuda.synchronize()
    assert not r.h[0].any() and not r.y[0].any() and not r.q_scale[0].any() and not r.x8_scale[0].any()
    assert r.y[1].isnan().all() and (r.q_scale[1] == 255).all() and r.x8_scale[1].tolist()[1] == 255
    # an infinite x: 1 / sqrt(inf) = 0 leaves the other values 0, its own NaN
    assert r.h[2, 3].isnan() and r.y[2].isnan().all()
    assert torch.equal(r.h[2, 4:].cpu(), (d["residual"][2, 4:].float() * d["residual_scale"]).bfloat16())
    assert r.h[3, 5].isinf() and r.y[3, 5].isnan() and not r.y[3, 6:].any()
    assert r.h[4, 7].isnan() and r.h[4, 8:].isfinite().all()
    sub = {k: v if v is None or k in ("post_gamma", "pre_gamma", "residual_scale") else v[5:] for k, v in d.items()}
    sub["gate"] = d["gate"][5:].clone()
    one = moe.sandwich_norm(**{k: cuda(v) for k, v in sub.items()}, out8="ocp")     # one row: a channel's gate
    assert same(r.h[5:], one.h) and same(r.q[5:], one.q)


# ------------------------------------------------------------------ gradient
def sandwich_tolerances(dh, dy, x, h, r1, r2, post, pre, gate, act, residual, scale):
    """What the operator's fp32 sums and products may be off by, from above (u8 = 2^-21: up to 8 roundings of a
    product or of a fused addition). With H = h r2, X = x r1, v = pre dy, w = post g:
    c2 = mean(v H) is off by S mean|v H|, d = dh + r2 (v - H c2) by u8 of its terms and r2 |H| S mean|v H|;
    the second mean is taken as B - c2 C: S of B's and C's magnitudes and C times c2's error."""
    u8 = 2.0 ** -21
    T, K = x.shape
    z = np.zeros_like(x)
    g, dg = P.gate_values(gate, act)
    X = x * r1[:, None] if post is not None else x
    H = h * r2[:, None] if dy is not None else z
    v = dy * pre if dy is not None else z
    rr = r2[:, None] if dy is not None else 0.0
    m = lambda a: np.mean(a, axis=1, keepdims=True)
    c2 = rr * m(v * H)
    e_c2 = S * rr * m(np.abs(v * H)) + u8 * np.abs(c2)
    d0 = np.abs(0 if dh is None else dh) + np.abs(rr * v)
    d_mag = d0 + np.abs(c2 * H)
    e_d = u8 * d_mag + np.abs(H) * e_c2
    p = np.ones((1, 1)) if post is None else post
    w = np.abs(p * g)
    out = dict(pre_gamma=np.abs(0 if dy is None else dy) * np.abs(H), e_d=e_d)
    out["residual"] = abs(1.0 if scale is None else scale) * (e_d + u8 * d_mag)
    if residual is not None:
        out["residual_scale"] = np.sum(np.abs(residual) * (e_d + S * d_mag + (T / 152 + 64) * 2.0 ** -24 * d_mag))
    wX = w * np.abs(X)
    if post is None:
        out["x"] = np.abs(g) * e_d + u8 * np.abs(g) * d_mag
    else:
        e_dot = S * (m(wX * d0) + np.abs(c2) * m(wX * np.abs(H))) + e_c2 * m(wX * np.abs(H))
        dot = m(wX * d_mag)
        out["x"] = np.abs(r1[:, None]) * (w * (e_d + u8 * d_mag) + np.abs(X) * (e_dot + u8 * dot))
        out["post_gamma"] = np.abs(g) * np.abs(X) * (e_d + u8 * d_mag)
    n = np.abs(X * p)
    out["gate"] = np.abs(dg) * n * (e_d + u8 * d_mag)
    out["gate_row"] = np.sum(np.abs(dg) * n * (e_d + S * d_mag), axis=1, keepdims=True) + \
        np.abs(dg[:, :1]) * np.abs(e_c2) * np.sum(n * np.abs(H), axis=1, keepdims=True)
    # sums over rows: a CTA's run of rows, then the CTAs: at most T / 152 + 64 additions
    n_add = (T / 152 + 64) * 2.0 ** -24
    for name, mag in (("pre_gamma", out["pre_gamma"]), ("post_gamma", np.abs(g) * np.abs(X) * d_mag),
                      ("gate_col", np.abs(dg) * n * d_mag)):
        err = u8 * mag if name == "pre_gamma" else out["post_gamma" if name == "post_gamma" and post is not None else "gate"]
        out[name] = np.sum(err + n_add * mag, axis=0)
    return out


def make_backward(d, act, eps=1e-5, ck=None, seed=0, with_dh=True, with_dy=True):
    """(the call's keyword arguments on the CPU, the oracle's values of the same) from the forward's oracle."""
    o = oracle_forward(d, act, eps)
    T, K = d["x"].shape
    g = gen(seed + 1)
    call = dict(grad_h=(torch.randn(T, K, generator=g) * 0.1).bfloat16() if with_dh else None,
                grad_y=(torch.randn(T, K, generator=g) * 0.1).bfloat16() if with_dy else None,
                rstd=torch.from_numpy(np.stack((o["r1"], o["r2"]))).float(),
                post_gamma=d["post_gamma"], pre_gamma=d["pre_gamma"], gate=d["gate"], gate_act=act,
                residual=d["residual"] if d["residual_scale"] is not None else None, residual_scale=d["residual_scale"])
    h = torch.from_numpy(o["h"]).float()
    if ck is None:
        call.update(x=d["x"], h=h.bfloat16())
        x64, h64 = f64(d["x"]), f64(call["h"])
    else:
        def enc(v):
            q, s = P.mx8_encode(v, ck)
            return torch.from_numpy(q).float().to(torch.float8_e4m3fn), torch.from_numpy(s), \
                q * np.repeat(np.exp2(s.astype(np.float64) - 127), 32, 1)
        call["x"], call["x_scale"], x64 = enc(f64(d["x"]))
        call["h"], call["h_scale"], h64 = enc(o["h"])
    if not with_dy:
        h64 = np.zeros_like(x64)
    vals = dict(dh=f64(call["grad_h"]), dy=f64(call["grad_y"]), x=x64, h=h64, r1=f64(call["rstd"][0]),
                r2=f64(call["rstd"][1]), post_gamma=f64(d["post_gamma"]), pre_gamma=f64(d["pre_gamma"]),
                gate=f64(d["gate"]), act=act, residual=f64(call["residual"]), scale=f64(d["residual_scale"]))
    if vals["scale"] is not None:
        vals["scale"] = float(vals["scale"][0])
    return call, vals


def check_backward(moe, call, vals, **kw):
    r = moe.sandwich_norm_backward(**{k: v if isinstance(v, str) else cuda(v) for k, v in call.items()}, **kw)
    torch.cuda.synchronize()
    ref = P.sandwich_norm_backward(**vals)
    tol = sandwich_tolerances(*vals.values())

    def near(name, got, want, t, rounding=0.0):
        bad = ~(np.abs(f64(got) - want) <= t + rounding * np.abs(want) + TINY)
        assert not bad.any(), (name, np.argwhere(bad)[:4], f64(got)[bad][:4], want[bad][:4],
                               np.broadcast_to(t, want.shape)[bad][:4])

    near("x", r.x, ref["x"], tol["x"], BF)
    near("residual", r.residual, ref["residual"], tol["residual"], BF)
    for name in ("post_gamma", "pre_gamma"):
        assert (getattr(r, name) is None) == (vals[name] is None)
        if vals[name] is not None:
            near(name, getattr(r, name), ref[name], tol[name])
    if vals["gate"] is None:
        assert r.gate is None
    elif r.gate.dtype == torch.bfloat16:
        near("gate", r.gate, ref["gate"], tol["gate"], BF)
    elif r.gate.shape[0] == 1 and call["gate"].dtype == torch.bfloat16:
        near("gate", r.gate[0], ref["gate"].sum(0), tol["gate_col"])
    else:
        near("gate", r.gate, ref["gate"].sum(1, keepdims=True), tol["gate_row"])
    assert (r.residual_scale is None) == (vals["residual"] is None)
    if vals["residual"] is not None:
        near("residual_scale", r.residual_scale, np.array([ref["residual_scale"]]), tol["residual_scale"])
    return r


@pytest.mark.parametrize("T,K", SHAPES)
@pytest.mark.parametrize("gate,act", [(None, "linear"), ("channel", "linear"), ("token", "sigmoid"), ("full", "sigmoid"),
                                      ("full", "linear"), ("channel", "sigmoid"), ("token", "linear")])
def test_sandwich_gradient_matches_oracle(moe, T, K, gate, act):
    for i, ck in enumerate((None, "ocp")):
        d = rows(T, K, T + K + i, gate, scaled=i == 0)
        check_backward(moe, *make_backward(d, act, ck=ck, seed=K))


@pytest.mark.parametrize("post,pre", [(False, True), (True, False), (False, False)])
def test_sandwich_gradient_without_a_norm(moe, post, pre):
    for gate in (None, "channel", "token", "full"):
        for ck in (None, "nosat"):
            check_backward(moe, *make_backward(rows(33, 1056, 7, gate, post, pre), "sigmoid", ck=ck, with_dy=pre))


@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
def test_sandwich_gradient_of_one_output(moe, gate):
    check_backward(moe, *make_backward(rows(20, 320, 3, gate), "linear", with_dy=False))
    check_backward(moe, *make_backward(rows(20, 320, 4, gate), "linear", with_dh=False))
    call, vals = make_backward(rows(20, 320, 4, gate, pre=False, post=False), "linear", with_dy=False)
    call.update(h=None, rstd=None)
    check_backward(moe, call, vals)


def test_sandwich_gradient_one_side_in_8_bits(moe):
    for side in ("x", "h"):
        a, va = make_backward(rows(50, 640, 5, "token"), "sigmoid")
        b, vb = make_backward(rows(50, 640, 5, "token"), "sigmoid", ck="ocp")
        a[side], a[side + "_scale"], va[side] = b[side], b[side + "_scale"], vb[side]
        check_backward(moe, a, va)


def test_sandwich_gradient_where_the_first_mean_takes_all(moe):
    """A gradient of y along h: the norm's Jacobian leaves a small difference of large terms."""
    d = rows(40, 1024, 6, "channel", spread=0.0)
    call, vals = make_backward(d, "linear", with_dh=False)
    H = vals["h"] * vals["r2"][:, None] / vals["pre_gamma"]
    call["grad_y"] = torch.from_numpy(H).float().bfloat16()
    vals["dy"] = f64(call["grad_y"])
    check_backward(moe, call, vals)


def test_sandwich_gradient_from_what_the_forward_kept(moe):
    """The forward's own rstd, h, x8 and h8; and the gradient against differences of the float64 forward.

    The kept h is off by a relative 2^-8 (bf16) or half a step of its 8-bit code; with dH that error times
    r2, the formula's d moves by at most r2 (dH |mean(v H)| + |H| mean|v dH|) where the factors are kept."""
    d = rows(3, 64, 12, "channel", spread=0.2)
    g = gen(13)
    dh, dy = ((0.1 * torch.randn(3, 64, generator=g)).bfloat16() for _ in range(2))
    c = {k: cuda(v) for k, v in d.items()}
    r = moe.sandwich_norm(**c, gate_act="sigmoid", eps=1e-5, checkpoint8="nosat", rstd=True)
    args = dict(post_gamma=c["post_gamma"], pre_gamma=c["pre_gamma"], gate=c["gate"], gate_act="sigmoid",
                residual=c["residual"], residual_scale=c["residual_scale"])

    def loss(x):
        o = P.sandwich_norm(x, f64(d["residual"]), f64(d["post_gamma"]), f64(d["pre_gamma"]), f64(d["gate"]), "sigmoid",
                            float(d["residual_scale"][0]), 1e-5)
        return float(np.sum(f64(dh) * o["h"]) + np.sum(f64(dy) * o["y"]))

    x = f64(d["x"])
    want = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += 1e-6
        b[i] -= 1e-6
        want[i] = (loss(a) - loss(b)) / 2e-6
    o = oracle_forward(d, "sigmoid", 1e-5)
    r1, r2 = o["r1"][:, None], o["r2"][:, None]
    H, v = o["h"] * r2, f64(dy) * f64(d["pre_gamma"])
    m = lambda a: np.mean(a, axis=1, keepdims=True)
    w = np.abs(f64(d["post_gamma"]) * P.gate_values(f64(d["gate"]), "sigmoid")[0])
    for x8 in (False, True):
        if x8:   # x in 8 bits changes the point itself: the oracle's formula at that point, h in 8 bits
            kept = dict(x=r.x8, x_scale=r.x8_scale, h=r.h8, h_scale=r.h8_scale)
            dec = lambda q, s: f64(q) * np.repeat(np.exp2(f64(s) - 127), 32, 1)
            vals = dict(dh=f64(dh), dy=f64(dy), x=dec(r.x8, r.x8_scale), h=dec(r.h8, r.h8_scale), r1=f64(r.rstd[0]),
                        r2=f64(r.rstd[1]), post_gamma=f64(d["post_gamma"]), pre_gamma=f64(d["pre_gamma"]),
                        gate=f64(d["gate"]), act="sigmoid", residual=f64(d["residual"]),
                        scale=float(d["residual_scale"][0]))
            call = dict(grad_h=dh, grad_y=dy, rstd=r.rstd, **kept,
                        **{k: v if isinstance(v, str) else v for k, v in args.items()})
            check_backward(moe, call, vals)
            continue
        got = f64(moe.sandwich_norm_backward(dh.cuda(), dy.cuda(), c["x"], r.h, r.rstd, **args).x)
        dH = BF * np.abs(H)
        e_d = r2 * (dH * np.abs(m(v * H)) + np.abs(H) * m(np.abs(v) * dH))
        X = np.abs(x) * r1
        e_x = r1 * (w * e_d + X * m(w * X * e_d))
        fp32 = sandwich_tolerances(f64(dh), f64(dy), x, o["h"], o["r1"], o["r2"], f64(d["post_gamma"]),
                                   f64(d["pre_gamma"]), f64(d["gate"]), "sigmoid", None, None)["x"]
        assert np.all(np.abs(got - want) <= e_x * 1.01 + fp32 + BF * np.abs(want) + 1e-8)


def test_sandwich_gradient_no_rows(moe):
    d = {k: cuda(v) for k, v in rows(4, 320, 3, "channel").items()}
    e = torch.empty(0, 320, dtype=torch.bfloat16, device="cuda")
    r = moe.sandwich_norm_backward(e, e, e, e, torch.empty(2, 0, device="cuda"), d["post_gamma"], d["pre_gamma"],
                                   d["gate"], residual=e, residual_scale=d["residual_scale"])
    assert r.x.shape == (0, 320) and r.gate.shape == (1, 320)
    for t in (r.post_gamma, r.pre_gamma, r.gate, r.residual_scale):
        assert not t.any()


def test_sandwich_gradient_nan_stays_in_its_row_and_columns(moe):
    call, vals = make_backward(rows(12, 128, 14, "token"), "linear", ck="ocp")
    call["x_scale"] = call["x_scale"].clone()
    ref = check_backward(moe, call, vals)
    call["x_scale"][5, 2] = 255
    r = moe.sandwich_norm_backward(**{k: v if isinstance(v, str) else cuda(v) for k, v in call.items()})
    keep = [t for t in range(12) if t != 5]
    assert same(r.x[keep], ref.x[keep]) and same(r.residual, ref.residual) and same(r.gate[keep], ref.gate[keep])
    assert r.x[5].isnan().all() and r.gate[5].isnan().all()
    assert r.post_gamma[64:96].isnan().all() and same(r.post_gamma[:64], ref.post_gamma[:64])
    assert same(r.pre_gamma, ref.pre_gamma)


def test_sandwich_offsets_past_32_bits(moe):
    T, K = 140_000, 16384
    at = torch.tensor([0, 131071, 131072, 131073, T - 1], device="cuda")   # 131072 * 16384 = 2^31
    big = lambda: torch.empty(T, K, dtype=torch.bfloat16, device="cuda").normal_()
    x, res, gate = big(), big(), big()
    gamma = torch.ones(K, device="cuda").bfloat16()
    r = moe.sandwich_norm(x, res, gamma, gamma, gate=gate, rstd=True, checkpoint8="ocp")
    pick = lambda t: t[at].contiguous()
    s = moe.sandwich_norm(pick(x), pick(res), gamma, gamma, gate=pick(gate), rstd=True, checkpoint8="ocp")
    for name in ("y", "h", "x8", "x8_scale", "h8", "h8_scale"):
        assert same(pick(getattr(r, name).view(torch.uint8)), getattr(s, name).view(torch.uint8)), name
    assert same(r.rstd[:, at].contiguous(), s.rstd)
    del x, res
    b = moe.sandwich_norm_backward(r.h, None, r.x8, None, r.rstd, gamma, gamma, gate=gate, x_scale=r.x8_scale)
    c = moe.sandwich_norm_backward(s.h, None, s.x8, None, s.rstd, gamma, gamma, gate=pick(gate), x_scale=s.x8_scale)
    assert same(pick(b.x), c.x) and same(pick(b.residual), c.residual) and same(pick(b.gate), c.gate)
    del r, b, gate
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ the routers
def routing(T, E, k, seed, pad=0.1, spread=1.0):
    g = gen(seed)
    x = torch.randn(T, E, generator=g) * spread
    ids = torch.argsort(torch.rand(T, E, generator=g), 1)[:, :k].int()
    ids[torch.rand(T, generator=g) < pad] = -1
    ids[torch.rand(T, k, generator=g) < pad] = -1
    return x, ids.contiguous()


def check_balance(moe, x, ids, scoring, off=None, **kw):
    r = moe.router_balance(x.cuda(), ids.cuda(), scoring, None if off is None else torch.tensor(off).int().cuda(), **kw)
    torch.cuda.synchronize()
    o = P.router_balance(x.numpy(), ids.numpy(), scoring, off)
    assert np.array_equal(r.counts.cpu().numpy(), o["counts"])
    st = f64(r.stats)
    assert st[2] == o["stats"][2] and st[3] == o["stats"][3]
    # p 2^-18, the sum over tokens at most T / 8 / 32 + 64 additions for the sizes here, all non-negative
    rel = 2.0 ** -17
    assert np.all(np.abs(f64(r.prob) - o["prob"]) <= rel * o["prob"] + TINY)
    assert np.all(np.abs(f64(r.slope) - o["slope"]) <= 2.0 ** -22 * o["slope"])
    assert abs(st[0] - o["stats"][0]) <= 2 * rel * o["stats"][0]
    # z: a relative 2^-17 of lse^2 where |lse| >= 1; below, an absolute error of 2 |lse| 2^-18
    assert abs(st[1] - o["stats"][1]) <= rel * (o["stats"][1] + 1)
    return r, o


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 17, 3), (40, 128, 4), (333, 160, 6), (70, 1024, 32),
                                   (500, 40, 8), (64, 513, 2), (9, 257, 9)])
def test_balance_matches_oracle(moe, scoring, T, E, k):
    x, ids = routing(T, E, k, T + E)
    check_balance(moe, x, ids, scoring)
    cut = sorted(np.random.default_rng(T).integers(0, T + 1, 5).tolist())
    check_balance(moe, x, ids, scoring, [0] + cut + [T])
    check_balance(moe, x, ids, scoring, [T // 3] + [max(c, T // 3) for c in cut[:3]])     # rows in no sequence


def test_balance_sequences_of_every_length(moe):
    x, ids = routing(600, 24, 3, 5, pad=0.2)
    rng = np.random.default_rng(6)
    check_balance(moe, x, ids, "sigmoid", list(range(601)))                                # one token each
    check_balance(moe, x, ids, "softmax", sorted(rng.integers(0, 601, 2000).tolist()))     # mostly empty
    check_balance(moe, x, ids, "softmax", [0] * 500 + [7] + [600] * 100)
    check_balance(moe, x, ids, "sigmoid", sorted(rng.integers(0, 601, 100).tolist()))
    check_balance(moe, x, ids, "sigmoid", [600, 600])


def test_balance_masks_and_padding(moe):
    inf, nan = float("inf"), float("nan")
    x, ids = routing(12, 40, 4, 7, pad=0)
    x[0, :39] = -inf
    x[1] = -inf
    x[2, 3:30] = nan
    x[3] = nan
    x[4] = torch.finfo(torch.float32).min
    x[5, 8] = torch.finfo(torch.float32).min
    ids[6] = -1
    ids[7] = 40                # past the experts: as padding
    ids[8] = ids[8, 0].item()  # the same expert four times
    ids[9, 1:] = 2 ** 31 - 1
    ids[10] = -2 ** 31
    for scoring in ("softmax", "sigmoid"):
        # the lowest fp32 squares to infinity: that row's log-sum-exp is out of range, as the float64 one is not
        y = x.clone()
        y[4] = -30.0
        check_balance(moe, y, ids, scoring)
        check_balance(moe, y, ids, scoring, [0, 2, 4, 5, 12])
        r = moe.router_balance(x.cuda(), ids.cuda(), scoring)
        assert r.stats[1].isinf() and r.prob.isfinite().all() and r.stats[0].isfinite()
    z = torch.full((3, 5), -200.0)   # every sigmoid 0 in fp32: no probability, the routes still count
    r = moe.router_balance(z.cuda(), torch.zeros(3, 1, dtype=torch.int32).cuda(), "sigmoid")
    assert not r.prob.any() and r.counts[0, 0] == 3 and r.stats[0] == 0 and r.stats[2] == 3


def test_balance_no_rows_and_no_tokens(moe):
    r = moe.router_balance(torch.empty(0, 9, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert not any(t.any() for t in r)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    r = moe.router_balance(torch.empty(0, 9, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                           seq_offsets=off)
    assert r.counts.shape == (3, 9) and not any(t.any() for t in r)
    r = moe.router_balance(torch.randn(50, 9, device="cuda"), torch.full((50, 2), -1, dtype=torch.int32, device="cuda"))
    assert not any(t.any() for t in r)


def test_balance_many_rows(moe):
    """More rows than one tile holds for every CTA; counts and even scores are exact sums."""
    T = 304 * 2048 + 4099
    x = torch.zeros(T, 4, device="cuda")
    ids = (torch.arange(T, device="cuda") % 3).int()[:, None].contiguous()
    r = moe.router_balance(x, ids, "softmax")
    assert r.counts[0].tolist() == torch.bincount(ids.flatten().long(), minlength=4).tolist()
    assert torch.equal(r.prob.cpu(), torch.full((1, 4), 0.25)) and abs(float(r.stats[0]) - 1) <= 2.0 ** -21
    off = torch.tensor([5, 100, 300_000, T - 7], dtype=torch.int32, device="cuda")
    r = moe.router_balance(x, ids, "softmax", off)
    for i in range(3):
        a, b = int(off[i]), int(off[i + 1])
        assert r.counts[i].tolist() == torch.bincount(ids[a:b].flatten().long(), minlength=4).tolist()
    assert float(r.stats[2]) == T - 12 and float(r.stats[3]) == 3


def check_router_backward(moe, x, ids, scoring, renorm, off=None, losses=True, weights=True, seed=0, scale=1.7):
    g = gen(seed)
    dw = torch.randn(ids.shape, generator=g) if weights else None
    dl = torch.tensor([0.7, 0.05]) if losses else None
    offd = None if off is None else torch.tensor(off).int().cuda()
    kw, bal = {}, None
    if losses:
        b = moe.router_balance(x.cuda(), ids.cuda(), scoring, offd)
        kw = dict(grad_losses=dl.cuda(), stats=b.stats, slope=b.slope, seq_offsets=offd)
        bal = P.router_balance(x.numpy(), ids.numpy(), scoring, off)
    out = torch.full(x.shape, float("nan"), device="cuda")
    got = moe.router_backward(x.cuda(), ids.cuda(), cuda(dw), scoring, renormalise=renorm, route_scale=scale,
                              grad_logits=out, **kw)
    torch.cuda.synchronize()
    assert got is out
    ref, mag = P.router_backward(x.numpy(), ids.numpy(), f64(dw), scoring, renorm, scale, f64(dl), bal)
    bad = ~(np.abs(f64(got) - ref) <= 2.0 ** -16 * mag + TINY)
    assert not bad.any(), (np.argwhere(bad)[:4], f64(got)[bad][:4], ref[bad][:4], mag[bad][:4])
    return got


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 17, 3), (60, 128, 4), (120, 160, 6), (20, 1024, 32),
                                   (50, 40, 8), (30, 513, 2), (9, 257, 9)])
def test_router_backward_matches_oracle(moe, scoring, renorm, T, E, k):
    x, ids = routing(T, E, k, T + E + 1)
    check_router_backward(moe, x, ids, scoring, renorm)
    check_router_backward(moe, x, ids, scoring, renorm, [0, T // 4, T // 4, T // 2])
    check_router_backward(moe, x, ids, scoring, renorm, losses=False)
    check_router_backward(moe, x, ids, scoring, renorm, [T // 5, T], weights=False)


def test_router_backward_masks_padding_and_repeats(moe):
    inf, nan = float("inf"), float("nan")
    x, ids = routing(12, 40, 4, 8, pad=0)
    x[0, :39] = -inf
    x[1] = -inf
    x[2, 3:30] = nan
    x[3] = nan
    ids[5] = -1
    ids[6] = 40
    ids[7] = ids[7, 0].item()
    ids[8, 1:] = ids[8, 1].item()
    ids[9, 1:] = 2 ** 31 - 1
    x[10] *= 30
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = check_router_backward(moe, x, ids, scoring, renorm, [0, 3, 12])
            assert not got[[1, 3, 5, 6]].any() and not got[0, :39].any() and not got[2, 3:30].any()
    # NaN in the weights' gradient of slots that take no part
    dw = torch.randn(12, 4, generator=gen(1))
    clean = moe.router_backward(x.cuda(), ids.cuda(), dw.cuda(), "sigmoid")
    dw[5], dw[6], dw[9, 1:], dw[1] = nan, inf, nan, nan
    assert same(clean, moe.router_backward(x.cuda(), ids.cuda(), dw.cuda(), "sigmoid"))


def test_router_backward_scores_out_of_range(moe):
    """Chosen scores that are 0 in fp32 (a bias chose them): gradients 0, nothing divided by them."""
    x = torch.full((2, 8), -200.0)
    x[1, 0] = 0.0
    ids = torch.tensor([[1, 2], [3, 4]], dtype=torch.int32)
    dw = torch.tensor([[1.0, -2.0], [3.0, 4.0]])
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            g = moe.router_backward(x.cuda(), ids.cuda(), dw.cuda(), scoring, renormalise=renorm)
            assert g.isfinite().all()
            assert not g[1].any()
    # nearly even logits, as large as fp32 takes them
    y = torch.full((1, 8), 3e38)
    g = moe.router_backward(y.cuda(), ids[:1].cuda(), dw[:1].cuda(), "softmax")
    assert g.isfinite().all() and abs(float(g[0, 1]) - 0.75) < 1e-6 and abs(float(g[0, 2]) + 0.75) < 1e-6


def test_router_backward_of_the_routers_own_choice(moe):
    """Through router_scored: the gradient of its weights against differences of the float64 weights of its ids."""
    x = torch.randn(6, 32, generator=gen(9)) * 0.5
    bias = 0.1 * torch.randn(32, generator=gen(10))
    dw = torch.randn(6, 4, generator=gen(11))
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, w = moe.router_scored(x.cuda(), 4, scoring, bias.cuda(), 8, 4, renormalise=renorm, route_scale=2.5)
            got = f64(moe.router_backward(x.cuda(), ids, dw.cuda(), scoring, renormalise=renorm, route_scale=2.5))
            i = ids.cpu().numpy()
            assert np.allclose(P.router_weights(x.numpy(), i, scoring, renorm, 2.5), f64(w), rtol=2.0 ** -17)
            want, x64 = np.zeros((6, 32)), f64(x)
            for at in np.ndindex(6, 32):
                a, b = x64.copy(), x64.copy()
                a[at] += 1e-6
                b[at] -= 1e-6
                want[at] = np.sum(f64(dw) * (P.router_weights(a, i, scoring, renorm, 2.5)
                                             - P.router_weights(b, i, scoring, renorm, 2.5))) / 2e-6
            _, mag = P.router_backward(x.numpy(), i, f64(dw), scoring, renorm, 2.5)
            assert np.all(np.abs(got - want) <= 2.0 ** -16 * mag + 1e-8)


# ------------------------------------------------------------------ the combination's gradient
def check_combine(moe, T, K, k, seed, ids=None, base=0, experts=0, routes_too=True):
    g = gen(seed)
    dy = (0.1 * torch.randn(T, K, generator=g)).bfloat16()
    o = torch.randn(T * k, K, generator=g).bfloat16()
    w = torch.rand(T, k, generator=g)
    if ids is not None:   # rows of skipped routes may hold anything
        live = (ids >= base) & ((ids < base + experts) if experts else torch.tensor(True))
        o[~live.flatten()] = float("nan")
    dw, do = moe.combine_backward(dy.cuda(), o.cuda(), cuda(ids), w.cuda(), routes_too, base, experts)
    torch.cuda.synchronize()
    ref, mag, dref = P.combine_backward(f64(dy), f64(o).reshape(T, k, K), None if ids is None else ids.numpy(), f64(w),
                                        base, experts)
    # a lane's serial sum has at most 16384 / 32 terms: K / 32 + 16 additions
    assert np.all(np.abs(f64(dw) - ref) <= (K / 32 + 16) * 2.0 ** -24 * mag)
    if not routes_too:
        assert do is None
        return
    assert np.all(np.abs(f64(do).reshape(T, k, K) - dref) <= (BF + 2.0 ** -23) * np.abs(dref) + TINY)
    if ids is not None:
        assert not do.cpu()[~live.flatten()].any() and not dw.cpu()[~live].any()


@pytest.mark.parametrize("T,K,k", [(1, 32, 1), (1, 2880, 4), (5, 7168, 8), (3, 16384, 3), (40, 96, 32), (700, 256, 2),
                                   (2, 8160, 9)])
def test_combine_backward_matches_oracle(moe, T, K, k):
    check_combine(moe, T, K, k, T + K)
    check_combine(moe, T, K, k, T + K, routes_too=False)
    ids = torch.randint(-2, 12, (T, k), generator=gen(k), dtype=torch.int32)
    check_combine(moe, T, K, k, T + K, ids)
    check_combine(moe, T, K, k, T + K, ids, 3, 5)
    check_combine(moe, T, K, k, T + K, torch.full((T, k), -1, dtype=torch.int32))


def test_combine_backward_offsets_past_32_bits(moe):
    T, k, K = 17_000, 8, 16384                                   # 17000 * 8 * 16384 = 2.2e9
    o = torch.empty(T * k, K, dtype=torch.bfloat16, device="cuda").normal_()
    dy = torch.randn(T, K, device="cuda").bfloat16()
    w = torch.rand(T, k, device="cuda")
    dw, do = moe.combine_backward(dy, o, topk_weights=w, routes_too=True)
    at = torch.tensor([0, 16383, 16384, 16385, T - 1], device="cuda")
    pick = (at[:, None] * k + torch.arange(k, device="cuda")).flatten()
    a, b = moe.combine_backward(dy[at].contiguous(), o[pick].contiguous(), topk_weights=w[at].contiguous(), routes_too=True)
    assert same(dw[at], a) and same(do[pick], b)
    del o, do
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ calls
def calls(moe, T=300, K=640, E=48, k=4, S=5):
    """Every operator as a function of keyword arguments (stream, workspace) and the bytes of its scratch."""
    d = {n: cuda(v) for n, v in rows(T, K, 21, "full").items()}
    call, _ = make_backward(rows(T, K, 21, "full"), "sigmoid", ck="ocp")
    call = {n: v if isinstance(v, str) else cuda(v) for n, v in call.items()}
    x, ids = (t.cuda() for t in routing(T, E, k, 22))
    off = torch.tensor([0, 10, 11, 150, 290, T], dtype=torch.int32).cuda()
    b = moe.router_balance(x, ids, "sigmoid", off)
    dw, dl = torch.randn(T, k, generator=gen(23)).cuda(), torch.tensor([0.1, 0.01]).cuda()
    dy, o = torch.randn(T, K, generator=gen(24)).bfloat16().cuda(), torch.randn(T * k, K, generator=gen(25)).bfloat16().cuda()
    w = torch.rand(T, k, generator=gen(26)).cuda()
    return {
        "sandwich_norm": (lambda **kw: moe.sandwich_norm(**d, out8="ocp", checkpoint8="nosat", rstd=True, **kw), 0),
        "sandwich_norm_backward": (lambda **kw: moe.sandwich_norm_backward(**call, **kw),
                                   moe.sandwich_norm_backward_workspace_size(T, K)),
        "router_balance": (lambda **kw: moe.router_balance(x, ids, "sigmoid", off, **kw),
                           moe.router_balance_workspace_size(T, E, S)),
        "router_backward": (lambda **kw: moe.router_backward(x, ids, dw, "sigmoid", grad_losses=dl, stats=b.stats,
                                                             slope=b.slope, seq_offsets=off, **kw), 0),
        "combine_backward": (lambda **kw: moe.combine_backward(dy, o, ids, w, True, **kw), 0),
    }


NAMES = ["sandwich_norm", "sandwich_norm_backward", "router_balance", "router_backward", "combine_backward"]


def copies(r):
    return [None if t is None else t.clone() for t in (r if isinstance(r, tuple) else (r,))]


@pytest.mark.parametrize("op", NAMES)
def test_repeats_on_streams_and_in_a_graph(moe, op):
    f, n = calls(moe)[op]
    want = copies(f())
    torch.cuda.synchronize()
    ws = dict(workspace=torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")) if n else {}
    for _ in range(3):
        assert same(copies(f(**ws)), want)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = [f(stream=s) for s in (a, b, a, b)]            # two calls at once
    torch.cuda.synchronize()
    assert all(same(copies(g), want) for g in got)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one = f(**ws)
    with torch.cuda.graph(other):                        # a second graph on the same workspace
        two = f(**ws)
    for _ in range(3):
        for t in copies(one) + copies(two):
            pass
        for r in (one, two):
            for t in (r if isinstance(r, tuple) else (r,)):
                if t is not None:
                    t.view(torch.uint8).fill_(0xFF)
        if n:
            ws["workspace"].fill_(0xFF)
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        assert same(copies(one), want) and same(copies(two), want)


@pytest.mark.parametrize("op", [n for n in NAMES if n in ("sandwich_norm_backward", "router_balance")])
def test_scratch_writes_stay_inside(moe, op):
    f, n = calls(moe)[op]
    G = 4096
    buf = torch.full((n + 2 * G,), 0xA5, dtype=torch.uint8, device="cuda")
    f(workspace=buf[G:G + n])
    torch.cuda.synchronize()
    assert (buf[:G] == 0xA5).all() and (buf[-G:] == 0xA5).all()
    with pytest.raises(moe.MoEError):
        f(workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("op", NAMES)
def test_call_on_another_stream_allocates_there(moe, monkeypatch, op):
    f, _ = calls(moe)[op]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    seen = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (seen.append(torch.cuda.current_stream()), empty(*a, **k))[1])
    f(stream=side)
    assert seen and all(s == side for s in seen)
    torch.cuda.synchronize()


def test_refusals(moe):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    x, g = bf(4, 64), bf(64)
    for kw in (dict(gate=bf(2, 64)), dict(gate=bf(4, 32)), dict(gate=torch.zeros(4, 64, device="cuda")),
               dict(gate_act="relu"), dict(out8="x"), dict(checkpoint8="x"), dict(residual_scale=torch.zeros(2, device="cuda")),
               dict(post_gamma=bf(32)), dict(out8="ocp"), dict(out=bf(4, 64)), dict(residual_out=bf(4, 32))):
        with pytest.raises((ValueError, TypeError)):
            moe.sandwich_norm(x, x, **kw)
    with pytest.raises(moe.MoEError):
        moe.sandwich_norm(bf(4, 48), bf(4, 48))
    with pytest.raises(ValueError):
        moe.sandwich_norm(x[:, :32], x[:, :32])
    r = torch.ones(2, 4, device="cuda")
    for kw in (dict(grad_y=x, h=None), dict(grad_y=x, pre_gamma=None), dict(post_gamma=g, rstd=None),
               dict(residual=x), dict(x_scale=torch.zeros(4, 2, dtype=torch.uint8, device="cuda")),
               dict(h=None, h_scale=torch.zeros(4, 2, dtype=torch.uint8, device="cuda")),
               dict(grad_x=bf(4, 32)), dict(rstd=torch.ones(4, 2, device="cuda"), post_gamma=g)):
        with pytest.raises((ValueError, TypeError)):
            moe.sandwich_norm_backward(**{**dict(grad_h=x, grad_y=None, x=x, h=x, rstd=r, pre_gamma=g), **kw})
    l, ids = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for kw in (dict(scoring="x"), dict(seq_offsets=torch.zeros(1, dtype=torch.int32, device="cuda")),
               dict(seq_offsets=torch.zeros(3, dtype=torch.int64, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            moe.router_balance(l, ids, **kw)
    with pytest.raises(ValueError):
        moe.router_balance(l, ids[:3].contiguous())
    with pytest.raises(moe.MoEError):
        moe.router_balance(l, torch.zeros(4, 9, dtype=torch.int32, device="cuda"))
    for kw in (dict(), dict(grad_losses=torch.zeros(2, device="cuda")), dict(grad_weights=torch.zeros(4, 3, device="cuda"))):
        with pytest.raises(ValueError):
            moe.router_backward(l, ids, **kw)
    with pytest.raises(ValueError):
        moe.combine_backward(x, bf(8, 64))
    with pytest.raises(ValueError):
        moe.combine_backward(x, bf(9, 64), ids)
    with pytest.raises(ValueError):
        moe.combine_backward(x, bf(8, 64), ids, routes_too=True)
