"""Cases of the operators around the MoE layer: the residual addition with RMS norm and its 8-bit output
(``add_rmsnorm``), the router in the score domain (``router_scored``) and the shared MXFP4 projection with
per-request low-rank adapters (``linear``).

``run`` computes a case in plain torch operations in 32 bits, or, where ``own`` is true, by the calls that a
user makes of this package. ``exact`` states each operator in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
# E2M1 magnitudes of codes 0..7; codes 8..15 are their negatives
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E4M3_MAX = 448.0


# ---------------------------------------------------------------- the cases
def _norm(name, T, K, out8, residual=True, rule="ocp"):
    return {"name": name, "op": "add_rmsnorm", "T": T, "K": K, "out8": out8, "residual": residual, "rule": rule}


def _router(name, T, E, topk, scoring, n_group=1, topk_group=1, bias=False, renormalise=True, scale=1.0):
    return {"name": name, "op": "router_scored", "T": T, "E": E, "topk": topk, "scoring": scoring,
            "n_group": n_group, "topk_group": topk_group, "bias": bias, "renormalise": renormalise,
            "scale": scale}


def _linear(name, T, K, N, rank, adapters, mixed, x8):
    return {"name": name, "op": "linear", "T": T, "K": K, "N": N, "rank": rank, "adapters": adapters,
            "mixed": mixed, "x8": x8}


def listed():
    return [
        # one token of one request, the norm before a 2880-wide MoE layer
        _norm("norm_t1_k2880", 1, 2880, False),
        # a decode batch whose normed rows go on in 8 bits
        _norm("norm_t32_k7168_mx8", 32, 7168, True),
        # a ragged batch of prompts, scales that never saturate
        _norm("norm_t777_k2880_mx8", 777, 2880, True, rule="nosat"),
        # a prefill chunk of 8192 tokens
        _norm("norm_t8192_k6144_mx8", 8192, 6144, True),
        # one token, 256 experts in 8 groups, the balance bias steering the choice
        _router("router_t1_e256_grouped", 1, 256, 8, "sigmoid", 8, 4, True, True, 2.5),
        # a decode batch, softmax over 128 experts
        _router("router_t32_e128_softmax", 32, 128, 4, "softmax"),
        # an odd expert count, softmax weights that are not renormalised
        _router("router_t4099_e160_softmax", 4099, 160, 6, "softmax", 1, 1, False, False, 16.0),
        # a prefill chunk, 256 experts in 8 groups
        _router("router_t8192_e256_grouped", 8192, 256, 8, "sigmoid", 8, 4, True, True, 2.5),
        # one token of one request with its adapter
        _linear("linear_t1_k6144_r16", 1, 6144, 4096, 16, 4, True, False),
        # a decode batch of 32 requests, each with an adapter of its own
        _linear("linear_t32_k2880_r16_mx8", 32, 2880, 5760, 16, 48, True, True),
        # a few prompts of a ragged batch, adapters of a larger rank
        _linear("linear_t517_k7168_r64", 517, 7168, 4096, 64, 5, False, False),
        # a prefill chunk of several requests, some without an adapter
        _linear("linear_t8192_k6144_r16_mx8", 8192, 6144, 4096, 16, 12, False, True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["add_rmsnorm", "router_scored", "linear"])
    T = _log_int(rng, 1, 8192)
    if op == "add_rmsnorm":
        c = _norm("", T, _log_int(rng, 512, 6144, 32), rng.random() < 0.6, rng.random() < 0.8,
                  rng.choice(["ocp", "nosat"]))
    elif op == "router_scored":
        if rng.random() < 0.5:
            n_group = rng.choice([1, 4, 8])
            E = n_group * rng.randrange(8, 257 // n_group)
            tg = rng.randrange(max(1, n_group // 2), n_group + 1)
            c = _router("", T, E, rng.randrange(1, 9), "sigmoid", n_group, tg, rng.random() < 0.7,
                        rng.random() < 0.7, rng.choice([1.0, 2.5]))
        else:
            c = _router("", T, rng.randrange(16, 257), rng.randrange(1, 9), "softmax", 1, 1, False,
                        rng.random() < 0.5, rng.choice([1.0, 16.0]))
    else:
        K = _log_int(rng, 512, 7168, 64)
        N = _log_int(rng, 512, 5760, 8)
        T = min(T, int(8192 * 6144 * 4096 / (K * N)))
        c = _linear("", T, K, N, rng.choice([8, 16, 24, 32, 64]), rng.randrange(1, 49),
                    T <= 64 or rng.random() < 0.1, rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _row_ids(c, g):
    """The adapter of each token: one request a token (mixed), or the prompts of several requests one
    after the other; every seventh adapter number stands for a request without one (-1)."""
    T, L = c["T"], c["adapters"]
    if c["mixed"]:
        ids = torch.randint(0, L, (T,), generator=g, device=DEV)
    else:
        cut = torch.randint(0, T, (L,), generator=g, device=DEV)
        order = torch.randperm(L + 1, generator=g, device=DEV)
        seg = (torch.arange(T, device=DEV)[:, None] >= cut[None, :]).sum(1)
        ids = order[seg]
    return torch.where((ids % 7 == 6) | (ids >= L), torch.full_like(ids, -1), ids).to(torch.int32)


def prepare(case, seed):
    g, c = _gen(seed), case
    T = c["T"]
    s = {"case": dict(c)}
    if c["op"] == "add_rmsnorm":
        K = c["K"]
        # the layer's output beside a residual stream a few times larger, with a few outlier channels
        s["x"] = _randn(g, T, K).to(torch.bfloat16)
        if c["residual"]:
            chan = torch.exp(0.5 * _randn(g, K)) * 3
            s["res"] = (_randn(g, T, K) * chan).to(torch.bfloat16)
        s["gamma"] = (1 + 0.2 * _randn(g, K)).to(torch.bfloat16)
    elif c["op"] == "router_scored":
        # gate logits, and a bias that balancing has moved in steps of 1/1024
        s["logits"] = _randn(g, T, c["E"])
        if c["bias"]:
            s["bias"] = torch.randint(-200, 201, (c["E"],), generator=g, device=DEV).float() / 1024
    else:
        K, N, L, r = c["K"], c["N"], c["adapters"], c["rank"]
        x = _randn(g, T, K)
        if c["x8"]:
            s["x"], s["sx"] = _to_mx8(x, "ocp")
        else:
            s["x"] = x.to(torch.bfloat16)
        s["w"] = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["s"] = torch.randint(118, 125, (N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
        s["ids"] = _row_ids(c, g)
        s["a"] = (_randn(g, L, r, K) / math.sqrt(K)).to(torch.bfloat16)
        s["b"] = (0.3 * _randn(g, L, N, r)).to(torch.bfloat16)
        s["alpha"] = 1 + torch.rand(L, generator=g, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms, 32 bits
def _to_mx8(y, rule):
    """fp32 rows -> E4M3 values and their E8M0 scale bytes, one scale per 32 values: the exponent of the
    block's largest magnitude less 8, raised by one under "nosat" where that would saturate; finite rows."""
    T, K = y.shape
    b = y.view(T, K // 32, 32)
    amax = b.abs().amax(-1)
    X = torch.where(amax > 0, torch.frexp(amax).exponent.int() - 9, -127).clamp(-127, 127)
    if rule == "nosat":
        X = (X + (torch.ldexp(amax, -X) > E4M3_MAX).int()).clamp(-127, 127)
    q = torch.ldexp(b, -X[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(T, K), (X + 127).to(torch.uint8)


def _from_mx8(q, scale):
    T, K = q.shape
    v = q.float().view(T, K // 32, 32) * torch.ldexp(torch.ones_like(scale, dtype=torch.float32), scale.int() - 127)[..., None]
    return v.view(T, K)


def _dequant(w, s):
    N, half = w.shape
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    v = torch.stack((table[(w & 15).long()], table[(w >> 4).long()]), -1).view(N, half // 16, 32)
    return (v * torch.ldexp(torch.ones_like(s, dtype=torch.float32), s.int() - 127)[..., None]).view(N, 2 * half)


def _plain_norm(c, s):
    h = s["x"].float()
    out = {}
    if c["residual"]:
        h = h + s["res"].float()
        out["residual"] = h.to(torch.bfloat16)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["gamma"].float()
    out["y"] = y.to(torch.bfloat16)
    if c["out8"]:
        q, sc = _to_mx8(y, c["rule"])
        out["q"], out["scale"] = q, sc.view(torch.float8_e8m0fnu)
    return out


def _plain_router(c, s):
    x, k, G = s["logits"], c["topk"], c["n_group"]
    T, E = x.shape
    if c["scoring"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True)
    choice = score + s["bias"] if c["bias"] else score
    # without a bias the choice goes by the logits: the score grows with them
    key = choice if c["bias"] else x
    if G > 1:
        two = choice.view(T, G, E // G).sort(dim=-1, descending=True).values[..., :2].sum(-1)
        best = two.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = (best[:, :, None] == torch.arange(G, device=DEV)).any(1)
        key = key.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    ids = key.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renormalise"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": w * c["scale"]}


def _plain_linear(c, s):
    x = _from_mx8(s["x"], s["sx"]) if c["x8"] else s["x"].float()
    T, L, r, N = c["T"], c["adapters"], c["rank"], c["N"]
    y = x @ _dequant(s["w"], s["s"]).t()
    # every token with every adapter, the others' products masked out
    v = (x @ s["a"].float().view(L * r, -1).t()).view(T, L, r)
    mine = s["ids"][:, None] == torch.arange(L, device=DEV)
    v = torch.where(mine[..., None], v * s["alpha"][:, None], torch.zeros((), device=DEV))
    y = y + v.view(T, L * r) @ s["b"].float().transpose(1, 2).reshape(L * r, N)
    return {"y": y.to(torch.bfloat16)}


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if not own:
        return {"add_rmsnorm": _plain_norm, "router_scored": _plain_router, "linear": _plain_linear}[c["op"]](c, state)
    from mxfp4_mixture_experts_gb300 import moe
    if c["op"] == "add_rmsnorm":
        y, res, q, scale = moe.add_rmsnorm(state["x"], state["gamma"], state.get("res"), eps=EPS,
                                           out8=c["rule"] if c["out8"] else None)
        out = {"y": y}
        if c["residual"]:
            out["residual"] = res
        if c["out8"]:
            out["q"], out["scale"] = q, scale.view(torch.float8_e8m0fnu)
        return out
    if c["op"] == "router_scored":
        ids, w = moe.router_scored(state["logits"], c["topk"], c["scoring"], state.get("bias"), c["n_group"],
                                   c["topk_group"], renormalise=c["renormalise"], route_scale=c["scale"])
        return {"ids": ids, "weights": w}
    y = moe.linear(state["x"], state["w"], state["s"], state.get("sx"), adapter_ids=state["ids"],
                   adapter_a=state["a"], adapter_b=state["b"], adapter_scale=state["alpha"])
    return {"y": y}


def work(case):
    """Each input read once and each output written once. A linear case reads the adapters that its tokens
    can name at most (min(T, adapters) of them) and multiplies each token by its own alone."""
    c, T = case, case["T"]
    if c["op"] == "add_rmsnorm":
        K = c["K"]
        per = 2 + 2 + (4 if c["residual"] else 0) + (1 + 1 / 32 if c["out8"] else 0)
        return {"bytes": T * K * per + 2 * K, "flops": T * K * 5}
    if c["op"] == "router_scored":
        return {"bytes": T * (4 * c["E"] + 8 * c["topk"]) + (4 * c["E"] if c["bias"] else 0), "flops": T * c["E"] * 4}
    K, N, r = c["K"], c["N"], c["rank"]
    xb = T * K * (1 + 1 / 32) if c["x8"] else T * K * 2
    used = min(T, c["adapters"])
    return {"bytes": xb + N * K * (0.5 + 1 / 32) + used * (r * (K + N) * 2 + 4) + T * (2 * N + 4),
            "flops": 2 * T * (K * N + r * (K + N))}


# ---------------------------------------------------------------- the definitions in 64 bits
def _mx8_64(y, rule):
    T, K = y.shape
    b = y.reshape(T, K // 32, 32)
    top = b.abs().max(-1).values
    e = torch.floor(torch.log2(top.clamp_min(1e-300)))
    e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e)) - 8
    if rule == "nosat":
        e = e + (top * torch.exp2(-e) > 448).double()
    e = torch.where(top > 0, e, -127.0).clamp(-127, 127)
    v = (b * torch.exp2(-e)[..., None]).clamp(-448, 448)
    # nearest E4M3 value, ties to even: steps of 2^-9 below 2^-6, else of an eighth of the power of two below
    p = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(p - 3)
    return (torch.round(v / step) * step).reshape(T, K), torch.exp2(e)


def exact(case, seed):
    s, c = prepare(case, seed), case
    T = c["T"]
    if c["op"] == "add_rmsnorm":
        h = s["x"].double()
        out = {}
        if c["residual"]:
            h = h + s["res"].double()
            out["residual"] = h
        y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / c["K"] + EPS) * s["gamma"].double()
        out["y"] = y
        if c["out8"]:
            out["q"], out["scale"] = _mx8_64(y, c["rule"])
        return out
    if c["op"] == "router_scored":
        x, E, G = s["logits"].double(), c["E"], c["n_group"]
        p = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, -1)
        pick = p + s["bias"].double() if c["bias"] else p.clone()
        if G > 1:
            groups = pick.view(T, G, E // G).topk(min(2, E // G), -1).values.sum(-1)
            # a group stays where fewer than topk_group groups beat it
            beat = (groups[:, None, :] > groups[:, :, None]).sum(-1)
            pick = torch.where((beat < c["topk_group"]).repeat_interleave(E // G, 1), pick, -1e9)
        w = torch.take_along_dim(p, torch.argsort(pick, -1, descending=True)[:, :c["topk"]], 1)
        if c["renormalise"]:
            w = w / w.sum(-1, keepdim=True)
        return {"ids": None, "weights": w * c["scale"]}
    N, K = c["N"], c["K"]
    if c["x8"]:
        x = s["x"].double() * torch.exp2(s["sx"].double() - 127).repeat_interleave(32, 1)
    else:
        x = s["x"].double()
    nib = torch.empty(N, K, dtype=torch.long, device=DEV)
    nib[:, 0::2], nib[:, 1::2] = s["w"] % 16, torch.div(s["w"], 16, rounding_mode="floor")
    m, e = nib % 2, torch.div(nib % 8, 2, rounding_mode="floor")
    mag = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
    w = torch.where(nib >= 8, -mag, mag) * torch.exp2(s["s"].double() - 127).repeat_interleave(32, 1)
    y = x @ w.t()
    for j in range(c["adapters"]):
        rows = torch.nonzero(s["ids"] == j).flatten()
        if rows.numel():
            y[rows] += s["alpha"][j].double() * (x[rows] @ s["a"][j].double().t()) @ s["b"][j].double().t()
    return {"y": y}
