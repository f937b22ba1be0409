"""The operators around the layer against their float64 oracle, at the sizes,
masks and ranges where they can go wrong.

Tolerances, from the operators' own roundings (u = 2^-24):
* the residual stream is one fp32 addition and one rounding to bf16: bit-exact;
* y: the fp32 sum of squares (at most 64 serial additions a thread and 10 tree
  steps), its mean, rsqrtf (2 ulp) and two products stay under 2^-18 relative;
  the bf16 output (8 significant bits) adds its unit roundoff, 2^-8 relative;
* MXFP8: half a step of E4M3 around y, with y's 2^-18;
* router: fp32 scores are within 2^-21 of the 64-bit ones (expf 2 ulp, one
  addition, one division, softmax sums of up to 1024 terms in a tree), one more
  rounding for the bias; two experts closer than twice that may trade places;
* linear: one fp32 rounding per tensor-core step of 16 values of the
  reduction, at most 2^-23 of the sum of magnitudes each, the inner adapter
  product rounded to bf16 (2^-8 of its magnitude) and the output's 2^-8."""
import numpy as np
import pytest
import torch

from oracle import mxfp4_moe_oracle as O
from oracle import operators_oracle as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    from mxfp4_mixture_experts_gb300 import moe
    return moe


def bits(t):
    return t.detach().cpu().view(torch.int16).numpy().view(np.uint16)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ add_rmsnorm
def check_norm(moe, x, gamma, res, eps, rule, in_place=None):
    xd, gd = x.cuda(), gamma.cuda()
    rd = None if res is None else res.cuda()
    ro = {None: None, "x": xd, "residual": rd}[in_place]
    out, ho, q, s = moe.add_rmsnorm(xd, gd, rd, eps=eps, out8=rule, residual_out=ro)
    torch.cuda.synchronize()
    h, y = P.add_rmsnorm(bits(x), bits(gamma), eps, None if res is None else bits(res))
    if res is not None or in_place:
        assert np.array_equal(bits(ho), O.float_to_bf16_bits(h))
    err = np.abs(f64(out) - y)
    assert not np.any(err > np.abs(y) * (2.0 ** -8 + 2.0 ** -18) + 2.0 ** -133)
    if rule is None:
        assert q is None and s is None
        return
    T, K = y.shape
    scale = s.cpu().numpy().astype(np.int64)
    amax = np.abs(y).reshape(T, K // 32, 32).max(-1)
    lo = np.vectorize(lambda v: P.mx8_exponent(v, rule))(amax * (1 - 2.0 ** -18)) + 127
    hi = np.vectorize(lambda v: P.mx8_exponent(v, rule))(amax * (1 + 2.0 ** -18)) + 127
    assert np.all((scale == lo) | (scale == hi))
    f = np.exp2(np.repeat(scale, 32, 1) - 127.0)
    v = np.abs(y) / f
    got = f64(q)
    _, e = np.frexp(np.minimum(v * (1 + 2.0 ** -18), 448.0))
    half = np.exp2(np.maximum(e - 1, -6) - 4.0)
    err = np.abs(got - np.sign(y) * np.minimum(v, 448.0))
    assert np.all(err <= half + v * 2.0 ** -18)
    if rule == "nosat":
        assert np.all(v <= 448 * (1 + 2.0 ** -17))


@pytest.mark.parametrize("T,K", [(1, 32), (1, 2880), (3, 64), (2, 7168), (5, 8160), (2, 8192),
                                 (2, 8224), (1, 16384), (33, 1056), (300, 96)])
@pytest.mark.parametrize("rule", [None, "ocp", "nosat"])
def test_add_rmsnorm_matches_oracle(moe, T, K, rule):
    g = gen(T * 7 + K)
    x = torch.randn(T, K, generator=g).bfloat16()
    res = (torch.randn(T, K, generator=g) * 4).bfloat16()
    gamma = (1 + 0.3 * torch.randn(K, generator=g)).bfloat16()
    check_norm(moe, x, gamma, res, 1e-5, rule)
    check_norm(moe, x, gamma, None, 1e-6, rule)


@pytest.mark.parametrize("in_place", ["x", "residual"])
def test_add_rmsnorm_in_place(moe, in_place):
    g = gen(5)
    x, res = (torch.randn(40, 2880, generator=g).bfloat16() for _ in range(2))
    check_norm(moe, x, torch.ones(2880).bfloat16(), res, 1e-5, "ocp", in_place)


def test_add_rmsnorm_block_ranges_and_saturation(moe):
    """Blocks at their own powers of two, and amax just under, at and above 448 * 2^X."""
    g = gen(6)
    K = 1024
    x = torch.randn(8, K, generator=g) * torch.pow(2.0, torch.randint(-30, 10, (8, K // 32), generator=g).float()).repeat_interleave(32, 1)
    x[1] = 1.0
    x[1, ::32] = 1.75
    x[2, ::32] = 1.7578125
    x[3] = 0
    x[3, 32:64] = 5.0
    for rule in ("ocp", "nosat"):
        check_norm(moe, x.bfloat16(), torch.ones(K).bfloat16(), None, 1e-5, rule)


def test_add_rmsnorm_zero_rows_and_nonfinite_rows(moe):
    x = torch.randn(4, 96, generator=gen(8)).bfloat16()
    x[0] = 0
    x[1, 40] = float("nan")
    x[2, 3] = float("inf")
    out, h, q, s = moe.add_rmsnorm(x.cuda(), torch.ones(96).bfloat16().cuda(), None, out8="ocp")
    torch.cuda.synchronize()
    assert not out[0].any() and not q[0].float().any() and not s[0].any()
    assert out[1].isnan().all() and (s[1] == 255).all() and not q[1].float().any()
    # 1 / sqrt(inf) = 0: finite values become 0, inf * 0 is NaN
    assert out[2, 3].isnan() and s[2, 0] == 255 and not out[2, 4:].any()
    ref = moe.add_rmsnorm(x[3:].cuda(), torch.ones(96).bfloat16().cuda(), None, out8="ocp")
    assert torch.equal(out[3:].view(torch.int16), ref[0].view(torch.int16))
    assert torch.equal(q[3:].view(torch.uint8), ref[2].view(torch.uint8))


def test_add_rmsnorm_outputs_alone_and_empty(moe):
    x = torch.randn(7, 320, generator=gen(9)).bfloat16().cuda()
    gamma = torch.ones(320).bfloat16().cuda()
    a = moe.add_rmsnorm(x, gamma, x, out8="ocp")
    b = moe.add_rmsnorm(x, gamma, x, out8="ocp", bf16=False)
    assert b[0] is None and torch.equal(a[2].view(torch.uint8), b[2].view(torch.uint8))
    assert torch.equal(a[3], b[3])
    e = moe.add_rmsnorm(x[:0], gamma, x[:0], out8="ocp")
    assert e[0].shape == (0, 320) and e[3].shape == (0, 10)
    with pytest.raises(ValueError):
        moe.add_rmsnorm(x[:, :160], gamma[:160])            # rows that are not contiguous
    with pytest.raises(moe.MoEError):
        moe.add_rmsnorm(x[:, :48].contiguous(), gamma[:48].contiguous())


# ------------------------------------------------------------------ router_scored
DELTA = 2.0 ** -21


def check_router(moe, logits, k, scoring, bias=None, **kw):
    ids, w = moe.router_scored(logits.cuda(), k, scoring, None if bias is None else bias.cuda(), **kw)
    torch.cuda.synchronize()
    ids, w = ids.cpu().numpy().astype(np.int64), w.cpu().numpy().astype(np.float64)
    x = logits.numpy()
    rid, rw, key = P.router_scored(x, k, scoring, None if bias is None else bias.numpy(), **kw)
    scale, renorm = kw.get("route_scale", 1.0), kw.get("renormalise", True)
    s = P.router_scores(x, scoring)
    swapped = 0
    for t in range(len(x)):
        if not np.array_equal(ids[t], rid[t]):
            assert bias is not None or kw.get("n_group", 1) > 1, "without a bias the logits decide exactly"
            swapped += 1
            got = ids[t]
            assert np.array_equal(got >= 0, rid[t] >= 0) and len(set(got)) == k
            c = np.where(np.isinf(key[t]), -np.inf, key[t])
            top = np.sort(c)[::-1][:k]
            tol = 2 * DELTA * max(1.0, np.abs(top[np.isfinite(top)]).max())
            assert np.all(np.abs(c[got] - top) <= tol), (t, got, rid[t])
        live = ids[t] >= 0
        want = np.where(live, s[t][ids[t]], 0.0)
        if renorm:
            want = want / want.sum() if want.sum() > 0 else want * 0
        assert np.all(np.abs(w[t] - want * scale) <= 2.0 ** -20 * np.abs(want * scale) + 1e-37)
    assert swapped <= max(1, len(x) // 500)
    return ids, w


@pytest.mark.parametrize("T,E,k,scoring,bias,kw", [
    (1, 256, 8, "sigmoid", True, dict(n_group=8, topk_group=4, route_scale=2.5)),
    (500, 256, 8, "sigmoid", True, dict(n_group=8, topk_group=4, route_scale=2.5)),
    (300, 256, 8, "sigmoid", False, dict(n_group=8, topk_group=3)),
    (33, 160, 6, "softmax", False, dict(renormalise=False, route_scale=16.0)),
    (300, 160, 6, "softmax", True, {}),
    (64, 128, 4, "softmax", False, {}),
    (40, 1024, 32, "sigmoid", True, dict(n_group=32, topk_group=32)),
    (40, 1024, 32, "softmax", False, dict(n_group=32, topk_group=1)),
    (17, 9, 9, "sigmoid", True, {}),
    (17, 9, 3, "sigmoid", True, dict(n_group=9, topk_group=3)),        # groups of one expert
    (50, 90, 5, "sigmoid", True, dict(n_group=6, topk_group=2, group_top=1)),
    (50, 72, 5, "softmax", True, dict(n_group=3, topk_group=2, renormalise=False)),
    (5, 1, 1, "softmax", False, {}),
    (9, 33, 32, "sigmoid", False, {}),
    (12, 520, 7, "sigmoid", True, dict(n_group=5, topk_group=2)),
])
def test_router_scored_matches_oracle(moe, T, E, k, scoring, bias, kw):
    g = gen(T * 13 + E + k)
    logits = torch.randn(T, E, generator=g) * 2
    b = 0.3 * torch.randn(E, generator=g) if bias else None
    check_router(moe, logits, k, scoring, b, **kw)


def test_router_scored_ties_to_the_lower_index(moe):
    g = gen(3)
    logits = torch.round(torch.randn(64, 256, generator=g) * 2) / 2
    logits[0] = 0.25
    logits[1, ::3] = 30.0           # sigmoids that round to 1: the logits decide
    logits[2, ::3] = torch.arange(86).float() + 30
    logits[3, 5], logits[3, 7] = -0.0, 0.0
    logits[3, :5] = -1.0
    logits[3, 8:] = -1.0
    logits[3, 6] = -1.0
    for scoring in ("softmax", "sigmoid"):
        for kw in ({}, dict(n_group=4, topk_group=4)):
            ids, _ = check_router(moe, logits, 8, scoring, **kw)
            assert list(ids[0]) == list(range(8))
            assert list(ids[1]) == [0, 3, 6, 9, 12, 15, 18, 21]
            assert list(ids[2]) == [255 - 3 * i for i in range(8)]
            assert list(ids[3, :2]) == [5, 7]
    ids, _ = check_router(moe, logits[:1], 8, "sigmoid", torch.zeros(256), n_group=8, topk_group=2)
    assert list(ids[0]) == list(range(8))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_router_scored_masked_experts(moe, scoring):
    """Experts out by -inf or NaN, by a -inf or NaN bias, groups and rows left empty, fp32's lowest value."""
    inf, nan = float("inf"), float("nan")
    x = torch.randn(8, 64, generator=gen(4))
    x[1, 8:] = -inf                 # 8 left
    x[2, 2:] = nan                  # 2 left for 4 slots
    x[3] = -inf
    x[4] = nan
    x[5, :63] = torch.finfo(torch.float32).min
    x[6, 3] = inf
    x[7, 32:] = -inf                # half the groups empty
    for kw in ({}, dict(n_group=8, topk_group=4), dict(n_group=8, topk_group=4, group_top=1)):
        ids, w = check_router(moe, x, 4, scoring, **kw)
        assert list(ids[2, 2:]) == [-1, -1] and not w[2, 2:].any()
        assert (ids[3] == -1).all() and (ids[4] == -1).all() and not w[3:5].any()
        assert np.isfinite(w).all()
        b = torch.zeros(64)
        b[0], b[1] = -inf, nan
        b[9] = torch.finfo(torch.float32).min
        ids, w = check_router(moe, x, 4, scoring, b, **kw)
        assert not np.isin(ids, [0, 1]).any() and (ids[2] == -1).all()


def test_router_scored_feeds_the_layer_with_padding(moe):
    """Slots without an expert are padding to the layer: an all-masked row gives a zero row."""
    g = gen(10)
    x = torch.randn(3, 8, generator=g)
    x[1] = -float("inf")
    ids, w = moe.router_scored(x.cuda(), 2, "sigmoid")
    h = torch.randn(3, 128, generator=g).bfloat16().cuda()
    w13 = torch.randint(0, 256, (8, 128, 64), generator=g, dtype=torch.uint8).cuda()
    s13 = torch.randint(118, 125, (8, 128, 4), generator=g, dtype=torch.uint8).cuda()
    w2 = torch.randint(0, 256, (8, 128, 32), generator=g, dtype=torch.uint8).cuda()
    s2 = torch.randint(118, 125, (8, 128, 2), generator=g, dtype=torch.uint8).cuda()
    y = moe.forward(h, ids, w, w13, s13, w2, s2)
    torch.cuda.synchronize()
    assert not y[1].any() and y[0].any() and y[2].any()


def test_router_scored_empty_and_refused(moe):
    ids, w = moe.router_scored(torch.empty(0, 16, device="cuda"), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    with pytest.raises(moe.MoEError):
        moe.router_scored(torch.zeros(2, 16, device="cuda"), 4, n_group=3)
    with pytest.raises(ValueError):
        moe.router_scored(torch.zeros(2, 16, device="cuda"), 4, "softmax_topk")
    with pytest.raises(ValueError):
        moe.router_scored(torch.zeros(16, 4, device="cuda").t(), 4)


# ------------------------------------------------------------------ linear
def make_linear(T, K, N, rank, L, x8, seed, ids="random", moe=None, x=None):
    g = gen(seed)
    d = {}
    x = torch.randn(T, K, generator=g) if x is None else x
    if x8:
        q, s = P.mx8_encode(x.double().numpy())
        d["x"] = torch.from_numpy(q).to(torch.float8_e4m3fn)
        d["x_scale"] = torch.from_numpy(s)
        d["x64"] = q * np.repeat(np.exp2(s.astype(np.float64) - 127), 32, 1)
    else:
        d["x"] = x.bfloat16()
        d["x64"] = f64(d["x"])
    d["w"] = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    d["s"] = torch.randint(115, 126, (N, K // 32), generator=g, dtype=torch.uint8)
    if rank:
        d["adapter_a"] = (torch.randn(L, rank, K, generator=g) / K ** 0.5).bfloat16()
        d["adapter_b"] = torch.randn(L, N, rank, generator=g).bfloat16()
        d["adapter_scale"] = 0.5 + torch.rand(L, generator=g)
        if ids == "random":
            d["adapter_ids"] = torch.randint(-1, L + 1, (T,), generator=g, dtype=torch.int32)
        elif ids == "runs":
            d["adapter_ids"] = (torch.arange(T) * (L + 1) // max(T, 1) - 1).to(torch.int32)
        else:
            d["adapter_ids"] = torch.full((T,), ids, dtype=torch.int32)
    return d


def call_linear(moe, d, **kw):
    a = {k: v.cuda() for k, v in d.items() if k != "x64"}
    return moe.linear(a.pop("x"), a.pop("w"), a.pop("s"), a.pop("x_scale", None), **a, **kw)


def check_linear(moe, d, rows=None, **kw):
    status = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    y = call_linear(moe, d, status=status, **kw)
    torch.cuda.synchronize()
    ids = d.get("adapter_ids")
    L = d["adapter_a"].shape[0] if ids is not None else 0
    assert status.tolist() == [int((ids >= L).sum()) if ids is not None else 0, 0, 0, 0]
    sel = np.arange(y.shape[0]) if rows is None else np.asarray(rows)
    K = d["x64"].shape[1]
    ref, mag, low = P.linear(d["x64"][sel], d["w"].numpy(), d["s"].numpy(),
                             None if ids is None else ids.numpy()[sel],
                             None if ids is None else bits(d["adapter_a"]),
                             None if ids is None else bits(d["adapter_b"]),
                             None if ids is None else d["adapter_scale"].numpy())
    got = f64(y)[sel]
    tol = 2.0 ** -8 * np.abs(ref) + (K / 16 + 16) * 2.0 ** -23 * (mag + low) + 2.0 ** -8 * 1.01 * low + 1e-37
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5])
    return y


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("T,K,N,rank,L", [
    (1, 64, 8, 8, 1), (1, 2880, 5760, 16, 3), (2, 128, 136, 24, 5), (5, 192, 1032, 64, 4),
    (16, 320, 264, 16, 40), (17, 64, 128, 256, 3), (32, 1024, 512, 32, 32), (33, 448, 392, 40, 7),
    (64, 512, 256, 16, 64), (100, 320, 648, 8, 11), (129, 256, 384, 128, 6), (256, 128, 128, 16, 300),
    (257, 704, 520, 96, 9), (700, 576, 264, 16, 20),
])
def test_linear_matches_oracle(moe, T, K, N, rank, L, x8):
    check_linear(moe, make_linear(T, K, N, rank, L, x8, T + K + N))


@pytest.mark.parametrize("T,K,N", [(1, 64, 8), (3, 2880, 128), (31, 6144, 264), (200, 192, 1000),
                                   (513, 128, 136)])
@pytest.mark.parametrize("x8", [False, True])
def test_linear_without_adapters(moe, T, K, N, x8):
    check_linear(moe, make_linear(T, K, N, 0, 0, x8, T + N))


@pytest.mark.parametrize("T,ids", [(20, -1), (20, 3), (20, 99), (300, "runs"), (300, -1), (300, 0),
                                   (1500, "runs")])
def test_linear_adapter_patterns(moe, T, ids):
    """No adapter at all, one for all, ids past the end, the runs of whole prompts."""
    d = make_linear(T, 256, 328, 16, 6, False, 31, ids)
    y = check_linear(moe, d)
    if ids in (-1, 99):
        plain = {k: v for k, v in d.items() if not k.startswith("adapter")}
        assert torch.equal(y, call_linear(moe, plain))


def test_linear_larger_rows_sampled(moe):
    d = make_linear(2100, 2880, 776, 32, 12, True, 5, "runs")
    check_linear(moe, d, rows=[0, 1, 127, 128, 255, 256, 257, 511, 512, 1000, 2047, 2048, 2099])
    d = make_linear(1025, 7168, 264, 64, 40, False, 6)
    check_linear(moe, d, rows=[0, 31, 32, 255, 256, 700, 1023, 1024])


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("rank", [8, 32, 40, 64, 72, 96, 136, 256])
@pytest.mark.parametrize("T", [4, 16, 20, 130])
def test_linear_ranks_with_k_in_parts(moe, T, rank, x8):
    """K split over clusters of the adapters' first product, ranks of one, two and more passes."""
    check_linear(moe, make_linear(T, 4096, 136, rank, 5, x8, 700 + T + rank))


@pytest.mark.parametrize("N", [4800, 4864, 9728, 10240])
def test_linear_few_free_sms(moe, N):
    """Outputs that leave the kernel before the projection few SMs, none, or half of each."""
    for T in (3, 16):
        check_linear(moe, make_linear(T, 1024, N, 64, 6, False, 800 + N + T), rows=[0, T - 1])


@pytest.mark.parametrize("ids", ["runs", "random"])
@pytest.mark.parametrize("K,x8", [(64, False), (192, True), (320, False)])
def test_linear_many_tiles_per_pair(moe, ids, K, x8):
    """More tiles than CTA pairs: each pair goes through several, with other adapters in each; K of one
    stage, of one and a half, and of a number of stages that the dequantising groups do not divide."""
    d = make_linear(3000, K, 2600, 24, 20, x8, 90 + K, ids)
    rows = list(range(0, 3000, 97)) + [255, 256, 1499, 2998, 2999]
    y = check_linear(moe, d, rows=rows)
    part = {k: (v[1000:1600] if k in ("x", "x_scale", "adapter_ids", "x64") else v) for k, v in d.items()}
    assert torch.equal(y[1000:1600], call_linear(moe, part))   # another tiling, the same sums


def test_linear_offsets_past_32_bits(moe):
    """2.46e9 outputs: rows around the 2^31st and the last ones."""
    T, K, N = 600_000, 64, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    d = make_linear(1, K, N, 16, 3, False, 91, 1)
    ids = torch.randint(-1, 3, (T,), generator=g, device="cuda", dtype=torch.int32)
    a = {k: v.cuda() for k, v in d.items() if k not in ("x64", "x", "adapter_ids")}
    y = moe.linear(x, a.pop("w"), a.pop("s"), adapter_ids=ids, **a)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 1, 524287, 524288, 524289, 599_998, 599_999])
    sub = dict(d, x=x[rows.cuda()].cpu(), adapter_ids=ids[rows.cuda()].cpu())
    sub["x64"] = f64(sub["x"])
    z = check_linear(moe, sub)
    assert torch.equal(y[rows.cuda()], z)
    del y
    torch.cuda.empty_cache()


def test_add_rmsnorm_offsets_past_32_bits(moe):
    T, K = 140_000, 16384
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").normal_()
    gamma = torch.ones(K).bfloat16()
    out, _, q, s = moe.add_rmsnorm(x, gamma.cuda(), None, out8="ocp")
    torch.cuda.synchronize()
    rows = torch.tensor([0, 131071, 131072, 131073, T - 1], device="cuda")   # 131072 * 16384 = 2^31
    ref = moe.add_rmsnorm(x[rows].contiguous(), gamma.cuda(), None, out8="ocp")
    assert torch.equal(out[rows], ref[0]) and torch.equal(s[rows], ref[3])
    assert torch.equal(q.view(torch.uint8)[rows], ref[2].view(torch.uint8))
    check_norm(moe, x[rows].cpu(), gamma, None, 1e-5, "ocp")
    del x, out, q, s
    torch.cuda.empty_cache()


def test_linear_rows_do_not_depend_on_the_batch(moe):
    """A token with the NaN or infinity of another one beside it keeps its values."""
    for T in (20, 300):
        d = make_linear(T, 320, 136, 16, 3, False, 40)
        y = call_linear(moe, d)
        x = d["x"].clone()
        x[7, 5] = float("nan")
        x[11, 300] = float("inf")
        e = dict(d, x=x)
        z = call_linear(moe, e)
        keep = [t for t in range(T) if t not in (7, 11)]
        assert torch.equal(y[keep], z[keep])
        assert z[7].isnan().all() and not z[11].isfinite().any()


def test_linear_adapter_of_another_token_may_hold_nan(moe):
    """An adapter that no token names is not read into any sum."""
    for T in (20, 300):
        d = make_linear(T, 320, 136, 16, 5, False, 41, 2)
        y = call_linear(moe, d)
        d["adapter_ids"][T // 2:] = 1
        d["adapter_a"][4] = float("nan")
        d["adapter_b"][4] = float("nan")
        d["adapter_b"][1] = float("nan")
        d["adapter_a"][1] = float("inf")
        z = call_linear(moe, d)
        assert torch.equal(y[:T // 2], z[:T // 2]) and z[T // 2:].isnan().all()


def test_linear_scale_extremes(moe):
    """E8M0 scales far from 127 on both sides, in weights and MXFP8 rows; byte 255 is NaN."""
    d = make_linear(24, 256, 136, 0, 0, True, 50)
    d["s"] = torch.randint(40, 60, d["s"].shape, generator=gen(1), dtype=torch.uint8)
    sx = torch.randint(170, 190, d["x_scale"].shape, generator=gen(2), dtype=torch.uint8)
    q = d["x"].double().numpy()
    d["x_scale"] = sx
    d["x64"] = q * np.repeat(np.exp2(sx.numpy().astype(np.float64) - 127), 32, 1)
    check_linear(moe, d)
    d["s"][5, 3] = 255
    d["x_scale"][2, 1] = 255
    y = call_linear(moe, d)
    assert y[:, 5].isnan().all() and y[2].isnan().all()
    rest = [t for t in range(24) if t != 2]
    assert y[rest][:, [n for n in range(136) if n != 5]].isfinite().all()


def test_linear_repeats_bit_for_bit_on_another_stream_and_in_a_graph(moe):
    for T, x8 in ((3, True), (40, False), (600, True)):
        d = make_linear(T, 1024, 520, 16, 9, x8, 60 + T)
        a = {k: v.cuda() for k, v in d.items() if k != "x64"}
        x, w, s, xs = a.pop("x"), a.pop("w"), a.pop("s"), a.pop("x_scale", None)
        n = moe.linear_workspace_size(T, 1024, 520, 16, x8)
        ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
        run = lambda out, **kw: moe.linear(x, w, s, xs, out=out, workspace=ws, **a, **kw)
        y = run(torch.empty(T, 520, dtype=torch.bfloat16, device="cuda")).clone()
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        z = torch.empty_like(y)
        run(z, stream=st)
        st.synchronize()
        assert torch.equal(y, z)
        z.fill_(float("nan"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(z)
        for _ in range(3):
            z.fill_(float("nan"))
            ws.fill_(0xFF)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, z)


@pytest.mark.parametrize("T", [1, 30, 200, 1030])
def test_linear_writes_stay_inside(moe, T):
    K, N, G = 320, 264, 4096
    d = make_linear(T, K, N, 24, 5, True, 70 + T)
    n = moe.linear_workspace_size(T, K, N, 24, True)
    ob = torch.full((T * N * 2 + 2 * G,), 0xA5, dtype=torch.uint8, device="cuda")
    wb = torch.full((n + 2 * G,), 0xA5, dtype=torch.uint8, device="cuda")
    out = ob[G:G + T * N * 2].view(torch.bfloat16).view(T, N)
    check_linear(moe, d, out=out, workspace=wb[G:G + n])
    for buf in (ob, wb):
        assert (buf[:G] == 0xA5).all() and (buf[-G:] == 0xA5).all()


def test_linear_empty_and_refused(moe):
    d = make_linear(4, 128, 64, 16, 2, False, 80)
    a = {k: v.cuda() for k, v in d.items() if k != "x64"}
    assert moe.linear(a["x"][:0], a["w"], a["s"]).shape == (0, 64)
    with pytest.raises(ValueError):
        moe.linear(a["x"], a["w"], a["s"], adapter_ids=a["adapter_ids"])
    with pytest.raises(ValueError):
        moe.linear(a["x"], a["w"], a["s"], adapter_a=a["adapter_a"])
    with pytest.raises(ValueError):
        moe.linear(a["x"][:, ::2], a["w"], a["s"])
    with pytest.raises(ValueError):
        moe.linear(a["x"], a["w"][:, :32].contiguous(), a["s"])
    with pytest.raises(moe.MoEError) as e:
        moe.linear(a["x"], a["w"], a["s"], adapter_ids=a["adapter_ids"], adapter_a=a["adapter_a"],
                   adapter_b=a["adapter_b"], workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.code == moe.ERR_WORKSPACE
