"""Cases of the operators that train what stands around the MXFP4 experts: the norms after and before a
block with the block's gate and the residual's scale (``sandwich_norm``), its gradient from bf16 or 8-bit
activations (``sandwich_norm_backward``), the balance losses and expert counts of a routing
(``router_balance``), the gradient of the router's logits (``router_backward``) and of the layer's
combination of its routes (``combine_backward``).

``run`` computes a case in plain torch operations in 32 bits, or, where ``own`` is true, by the calls that a
user makes of this package. ``exact`` states each operator in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
E4M3_MAX = 448.0


# ---------------------------------------------------------------- the cases
def _sandwich(name, T, K, gate, act, scaled, out8=None, checkpoint8=None, post=True, train=False):
    """gate: None, "channel" [1, K], "token" [T, 1] or "full" [T, K]; scaled: with a residual scale."""
    return {"name": name, "op": "sandwich_norm", "T": T, "K": K, "gate": gate, "act": act, "scaled": scaled,
            "out8": out8, "checkpoint8": checkpoint8, "post": post, "train": train}


def _sandwich_bwd(name, T, K, gate, act, scaled, checkpoint8=None, post=True):
    return {"name": name, "op": "sandwich_norm_backward", "T": T, "K": K, "gate": gate, "act": act,
            "scaled": scaled, "checkpoint8": checkpoint8, "post": post}


def _balance(name, T, E, topk, scoring, sequences):
    """sequences 0: the whole batch as one, without offsets."""
    return {"name": name, "op": "router_balance", "T": T, "E": E, "topk": topk, "scoring": scoring,
            "sequences": sequences}


def _router_bwd(name, T, E, topk, scoring, sequences, renormalise, scale):
    return {"name": name, "op": "router_backward", "T": T, "E": E, "topk": topk, "scoring": scoring,
            "sequences": sequences, "renormalise": renormalise, "scale": scale}


def _combine_bwd(name, T, K, topk, routes_too):
    return {"name": name, "op": "combine_backward", "T": T, "K": K, "topk": topk, "routes_too": routes_too}


def listed():
    return [
        # one token of one request between two 2880-wide blocks
        _sandwich("sandwich_t1_k2880", 1, 2880, None, "linear", False),
        # a decode batch with a gate for each token, whose normed rows go on in 8 bits
        _sandwich("sandwich_t32_k7168_mx8", 32, 7168, "token", "sigmoid", True, out8="nosat"),
        # a training batch that keeps 8-bit activations for its backward pass
        _sandwich("sandwich_t8192_k6144_ckpt8", 8192, 6144, "channel", "linear", False, checkpoint8="nosat",
                  train=True),
        # the gradient of a small ragged batch
        _sandwich_bwd("sandwich_bwd_t61_k2880", 61, 2880, "token", "sigmoid", False),
        # a few ragged prompts, a gate for each value, a trained residual scale
        _sandwich_bwd("sandwich_bwd_t777_k2880_full", 777, 2880, "full", "sigmoid", True),
        # the gradient of a training batch from its 8-bit activations
        _sandwich_bwd("sandwich_bwd_t8192_k6144_ckpt8", 8192, 6144, "channel", "linear", False,
                      checkpoint8="nosat"),
        # the counts of a decode batch, as a serving loop watches them
        _balance("balance_t32_e128_softmax", 32, 128, 4, "softmax", 0),
        # a training batch of twelve ragged sequences, each balanced by itself
        _balance("balance_t8192_e256_sigmoid", 8192, 256, 8, "sigmoid", 12),
        # a ragged batch, softmax weights that are not renormalised
        _router_bwd("router_bwd_t777_e160_softmax", 777, 160, 6, "softmax", 0, False, 16.0),
        # a training batch of twelve ragged sequences, renormalised sigmoid weights
        _router_bwd("router_bwd_t8192_e256_sigmoid", 8192, 256, 8, "sigmoid", 12, True, 2.5),
        # the routing weights' gradient of a small batch
        _combine_bwd("combine_bwd_t33_k2880_top4", 33, 2880, 4, False),
        # a training batch whose routes' own gradients go on into the experts
        _combine_bwd("combine_bwd_t4096_k6144_top8", 4096, 6144, 8, True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["sandwich_norm", "sandwich_norm_backward", "router_balance", "router_backward",
                     "combine_backward"])
    T = _log_int(rng, 1, 8192)
    if op.startswith("sandwich"):
        K = _log_int(rng, 512, 7168, 32)
        # the full gate, the residual and their gradients are further rows to move
        gate = rng.choice([None, "channel", "token", "full"])
        scaled = rng.random() < 0.5
        T = min(T, 8192 * 6144 // (K * (2 if gate == "full" or scaled else 1)))
        if T == 1 and gate == "full":
            gate = "channel"   # (one row of gates is a channel's)
        ck = rng.choice([None, "ocp", "nosat"])
        args = ("", T, K, gate, rng.choice(["linear", "sigmoid"]), scaled)
        if op == "sandwich_norm":
            train = ck is not None or rng.random() < 0.3
            o8 = None if ck is not None else rng.choice([None, "ocp", "nosat"])
            c = _sandwich(*args, out8=o8, checkpoint8=ck, post=rng.random() < 0.8, train=train)
        else:
            c = _sandwich_bwd(*args, checkpoint8=ck, post=rng.random() < 0.8)
    elif op == "combine_backward":
        K, k = _log_int(rng, 512, 7168, 32), rng.randrange(1, 9)
        c = _combine_bwd("", min(T, 4096 * 6144 * 8 // (K * k)), K, k, rng.random() < 0.5)
    else:
        E = rng.randrange(16, 257)
        S = rng.choice([0, 1, rng.randrange(2, 65)])
        args = ("", T, E, rng.randrange(1, 9), rng.choice(["softmax", "sigmoid"]), S)
        if op == "router_balance":
            c = _balance(*args)
        else:
            c = _router_bwd(*args, rng.random() < 0.6, rng.choice([1.0, 2.5]))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _norm_inputs(c, s, g):
    T, K = c["T"], c["K"]
    # a block's output beside a residual stream a few times larger, with a few outlier channels
    s["x"] = (_randn(g, T, K) * torch.exp(0.3 * _randn(g, T, 1))).to(torch.bfloat16)
    s["res"] = (_randn(g, T, K) * torch.exp(0.5 * _randn(g, K)) * 3).to(torch.bfloat16)
    s["g_post"] = (0.4 + 0.1 * _randn(g, K)).to(torch.bfloat16) if c["post"] else None
    s["g_pre"] = (1 + 0.2 * _randn(g, K)).to(torch.bfloat16)
    s["gate"] = None
    if c["gate"] == "channel":
        s["gate"] = (0.5 + 0.3 * _randn(g, 1, K)).to(torch.bfloat16)
    elif c["gate"] == "token":
        s["gate"] = _randn(g, T, 1)
    elif c["gate"] == "full":
        s["gate"] = _randn(g, T, K).to(torch.bfloat16)
    s["scale"] = 0.8 + 0.2 * torch.rand(1, generator=g, device=DEV) if c["scaled"] else None


def _routing(c, s, g):
    """Logits whose experts are not alike, the top k of their scores, rows of padding at the end of some
    sequences, and the sequences' offsets: lengths as ragged as they come, the last one may end early."""
    T, E, k = c["T"], c["E"], c["topk"]
    x = _randn(g, T, E) + 0.5 * _randn(g, E)
    s["logits"] = x
    ids = x.sort(dim=-1, descending=True, stable=True).indices[:, :k].to(torch.int32)
    if T > 1:
        pad = torch.rand(T, generator=g, device=DEV) < 0.03
        ids = torch.where(pad[:, None], torch.full_like(ids, -1), ids)
    s["ids"] = ids.contiguous()
    s["offsets"] = None
    if c["sequences"]:
        cut = torch.randint(0, T + 1, (c["sequences"],), generator=g, device=DEV).sort().values
        if c["sequences"] > 1:
            cut[-1] = max(T - 3, 0)
            cut = cut.sort().values
        else:
            cut[-1] = T
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), cut]).to(torch.int32)


def prepare(case, seed):
    g, c = _gen(seed), case
    T = c["T"]
    s = {"case": dict(c)}
    if c["op"] == "sandwich_norm":
        _norm_inputs(c, s, g)
    elif c["op"] == "sandwich_norm_backward":
        K = c["K"]
        _norm_inputs(c, s, g)
        s["dh"] = (1e-3 * _randn(g, T, K)).to(torch.bfloat16)
        s["dy"] = (1e-3 * _randn(g, T, K)).to(torch.bfloat16)
        # what the forward pass keeps
        r1, h, r2 = _forward(c, s)
        s["rstd"] = torch.stack((r1, r2))
        s["h"] = h.to(torch.bfloat16)
        if c["checkpoint8"]:
            s["x"], s["sx"] = _to_mx8(s["x"].float(), c["checkpoint8"])
            s["h"], s["sh"] = _to_mx8(h, c["checkpoint8"])
    elif c["op"] == "router_balance":
        _routing(c, s, g)
    elif c["op"] == "router_backward":
        _routing(c, s, g)
        s["dw"] = 1e-2 * _randn(g, T, c["topk"])
        # loss coefficients of 1e-2 and 1e-3, as the losses' own gradients
        s["dloss"] = torch.tensor([1e-2, 1e-3], device=DEV)
        s["stats"], _, _, s["slope"] = _balance_plain(c, s)
    else:
        K, k = c["K"], c["topk"]
        s["dy"] = (1e-2 * _randn(g, T, K)).to(torch.bfloat16)
        s["routes"] = _randn(g, T * k, K).to(torch.bfloat16)
        w = torch.rand(T, k, generator=g, device=DEV) + 0.1
        s["w"] = w / w.sum(-1, keepdim=True)
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


def _act(c, gate):
    if gate is None:
        return None
    gate = gate.float()
    return 1 / (1 + torch.exp(-gate)) if c["act"] == "sigmoid" else gate


def _forward(c, s):
    """Both norms' factors and the residual stream in 32 bits."""
    x = s["x"].float()
    r1 = torch.ones(c["T"], device=DEV)
    n = x
    if s["g_post"] is not None:
        r1 = torch.rsqrt(x.square().mean(-1) + EPS)
        n = x * r1[:, None] * s["g_post"].float()
    gate = _act(c, s["gate"])
    if gate is not None:
        n = n * gate
    h = s["res"].float()
    if s["scale"] is not None:
        h = h * s["scale"]
    h = h + n
    return r1, h, torch.rsqrt(h.square().mean(-1) + EPS)


def _plain_sandwich(c, s):
    r1, h, r2 = _forward(c, s)
    y = h * r2[:, None] * s["g_pre"].float()
    out = {"y": y.to(torch.bfloat16), "h": h.to(torch.bfloat16)}
    if c["out8"]:
        q, sc = _to_mx8(y, c["out8"])
        out["q"], out["scale"] = q, sc.view(torch.float8_e8m0fnu)
    if c["train"]:
        out["rstd"] = torch.stack((r1, r2))
    if c["checkpoint8"]:
        q, sc = _to_mx8(s["x"].float(), c["checkpoint8"])
        out["x8"], out["x8_scale"] = q, sc.view(torch.float8_e8m0fnu)
        q, sc = _to_mx8(h, c["checkpoint8"])
        out["h8"], out["h8_scale"] = q, sc.view(torch.float8_e8m0fnu)
    return out


def _plain_sandwich_bwd(c, s):
    x = _from_mx8(s["x"], s["sx"]) if c["checkpoint8"] else s["x"].float()
    h = _from_mx8(s["h"], s["sh"]) if c["checkpoint8"] else s["h"].float()
    r1, r2 = s["rstd"][0][:, None], s["rstd"][1][:, None]
    dy = s["dy"].float()
    hn = h * r2
    v = dy * s["g_pre"].float()
    dh = s["dh"].float() + r2 * (v - hn * (v * hn).mean(-1, keepdim=True))
    out = {"pre_gamma": (dy * hn).sum(0)}
    if s["scale"] is not None:
        out["residual_scale"] = (dh * s["res"].float()).sum().reshape(1)
        out["residual"] = (dh * s["scale"]).to(torch.bfloat16)
    else:
        out["residual"] = dh.to(torch.bfloat16)
    gate = _act(c, s["gate"])
    dn = dh if gate is None else dh * gate
    xn = x * r1 if c["post"] else x
    if c["post"]:
        u = dn * s["g_post"].float()
        out["post_gamma"] = (dn * xn).sum(0)
        out["x"] = (r1 * (u - xn * (u * xn).mean(-1, keepdim=True))).to(torch.bfloat16)
        n = xn * s["g_post"].float()
    else:
        out["x"] = dn.to(torch.bfloat16)
        n = x
    if gate is not None:
        d = dh * n
        if c["act"] == "sigmoid":
            d = d * gate * (1 - gate)
        if c["gate"] == "channel":
            out["gate"] = d.sum(0, keepdim=True)
        elif c["gate"] == "token":
            out["gate"] = d.sum(1, keepdim=True)
        else:
            out["gate"] = d.to(torch.bfloat16)
    return out


def _scores(c, x):
    if c["scoring"] == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _lse(x):
    m = x.amax(-1)
    return m + torch.log(torch.exp(x - m[:, None]).sum(-1))


def _member(c, s):
    """[S, T] truth values: the tokens of each sequence, rows of padding left out."""
    t = torch.arange(c["T"], device=DEV)
    live = (s["ids"] >= 0).any(-1)
    if s["offsets"] is None:
        return live[None]
    o = s["offsets"]
    return (t >= o[:-1, None]) & (t < o[1:, None]) & live


def _balance_plain(c, s):
    x, ids, E = s["logits"], s["ids"], c["E"]
    sc = _scores(c, x)
    p = sc / sc.sum(-1, keepdim=True)
    mine = _member(c, s)
    m = mine.float()
    hot = (ids[:, :, None] == torch.arange(E, device=DEV)).sum(1).float()
    counts = m @ hot
    n = mine.sum(-1).float()
    seen = n > 0
    one = torch.ones((), device=DEV)
    prob = (m @ p) / torch.where(seen, n, one)[:, None]
    total = counts.sum(-1)
    share = E * counts / torch.where(seen, total, one)[:, None]
    S = seen.sum().float()
    balance = (share * prob).sum() / torch.where(S > 0, S, one)
    tokens = n.sum()
    z = (_lse(x).square() * m.sum(0)).sum() / torch.where(tokens > 0, tokens, one)
    slope = share / torch.where(seen, n, one)[:, None]
    return torch.stack((balance, z, tokens, S)), counts.to(torch.int32), prob, slope


def _plain_balance(c, s):
    stats, counts, prob, slope = _balance_plain(c, s)
    return {"stats": stats, "counts": counts, "prob": prob, "slope": slope}


def _plain_router_bwd(c, s):
    x, ids, E = s["logits"], s["ids"], c["E"]
    sc = _scores(c, x)
    ok = ids >= 0
    col = ids.clamp_min(0).long()
    zero = torch.zeros((), device=DEV)
    dw = torch.where(ok, s["dw"], zero)
    chosen = torch.where(ok, sc.gather(1, col), zero)
    if c["renormalise"]:
        D = chosen.sum(-1, keepdim=True)
        q = torch.where(D > 0, chosen / D, zero)
        ds = torch.where(D > 0, (dw - (q * dw).sum(-1, keepdim=True)) / D, zero)
    else:
        ds = dw
    ds = c["scale"] * torch.where(ok, ds, zero)
    G = ((col[:, :, None] == torch.arange(E, device=DEV)) * ds[:, :, None]).sum(1)
    # the tokens' slopes, 0 for rows that no sequence counts
    m = _member(c, s).float()
    slope = (m.t() @ s["slope"]) * s["dloss"][0] / s["stats"][3].clamp_min(1)
    total = sc.sum(-1, keepdim=True)
    p = sc / total
    G = G + (slope - (p * slope).sum(-1, keepdim=True)) / total
    if c["scoring"] == "sigmoid":
        dx = G * sc * (1 - sc)
    else:
        dx = sc * (G - (sc * G).sum(-1, keepdim=True))
    e = torch.exp(x - x.amax(-1, keepdim=True))
    soft = e / e.sum(-1, keepdim=True)
    dz = 2 * s["dloss"][1] * _lse(x) * m.sum(0) / s["stats"][2].clamp_min(1)
    return {"logits": dx + soft * dz[:, None]}


def _plain_combine_bwd(c, s):
    T, K, k = c["T"], c["K"], c["topk"]
    dy = s["dy"].float()
    out = {"weights": (s["routes"].float().view(T, k, K) * dy[:, None]).sum(-1)}
    if c["routes_too"]:
        out["routes"] = (s["w"][:, :, None] * dy[:, None]).to(torch.bfloat16).view(T * k, K)
    return out


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    s = state
    if not own:
        return {"sandwich_norm": _plain_sandwich, "sandwich_norm_backward": _plain_sandwich_bwd,
                "router_balance": _plain_balance, "router_backward": _plain_router_bwd,
                "combine_backward": _plain_combine_bwd}[c["op"]](c, s)
    from mxfp4_mixture_experts_gb300 import moe
    if c["op"] == "sandwich_norm":
        r = moe.sandwich_norm(s["x"], s["res"], s["g_post"], s["g_pre"], gate=s["gate"], gate_act=c["act"],
                              residual_scale=s["scale"], eps=EPS, out8=c["out8"], checkpoint8=c["checkpoint8"],
                              rstd=c["train"])
        out = {"y": r.y, "h": r.h}
        if c["out8"]:
            out["q"], out["scale"] = r.q, r.q_scale.view(torch.float8_e8m0fnu)
        if c["train"]:
            out["rstd"] = r.rstd
        if c["checkpoint8"]:
            out["x8"], out["x8_scale"] = r.x8, r.x8_scale.view(torch.float8_e8m0fnu)
            out["h8"], out["h8_scale"] = r.h8, r.h8_scale.view(torch.float8_e8m0fnu)
        return out
    if c["op"] == "sandwich_norm_backward":
        r = moe.sandwich_norm_backward(s["dh"], s["dy"], s["x"], s["h"], s["rstd"], s["g_post"], s["g_pre"],
                                       gate=s["gate"], gate_act=c["act"],
                                       residual=s["res"] if c["scaled"] else None, residual_scale=s["scale"],
                                       x_scale=s.get("sx"), h_scale=s.get("sh"))
        out = {"x": r.x, "residual": r.residual, "pre_gamma": r.pre_gamma}
        if c["post"]:
            out["post_gamma"] = r.post_gamma
        if c["gate"]:
            out["gate"] = r.gate
        if c["scaled"]:
            out["residual_scale"] = r.residual_scale
        return out
    if c["op"] == "router_balance":
        r = moe.router_balance(s["logits"], s["ids"], c["scoring"], s["offsets"])
        return {"stats": r.stats, "counts": r.counts, "prob": r.prob, "slope": r.slope}
    if c["op"] == "router_backward":
        d = moe.router_backward(s["logits"], s["ids"], s["dw"], c["scoring"], renormalise=c["renormalise"],
                                route_scale=c["scale"], grad_losses=s["dloss"], stats=s["stats"],
                                slope=s["slope"], seq_offsets=s["offsets"])
        return {"logits": d}
    dw, dr = moe.combine_backward(s["dy"], s["routes"], topk_weights=s["w"], routes_too=c["routes_too"])
    return {"weights": dw, "routes": dr} if c["routes_too"] else {"weights": dw}


def work(case):
    """Each input read once and each output written once."""
    c, T = case, case["T"]
    mx = 33 / 32
    if c["op"].startswith("sandwich"):
        K = c["K"]
        per, row, once = 0, 0, 2 * K + (2 * K if c["post"] else 0)
        if c["op"] == "sandwich_norm":
            per = 2 + 2 + 2 + 2 + (mx if c["out8"] else 0) + (2 * mx if c["checkpoint8"] else 0)
            row = 8 if c["train"] else 0
            per, row, once = (per + (2 if c["gate"] == "full" else 0), row + (4 if c["gate"] == "token" else 0),
                              once + (2 * K if c["gate"] == "channel" else 0))
            return {"bytes": T * (K * per + row) + once, "flops": T * K * 10}
        per = 4 + 2 * (mx if c["checkpoint8"] else 2) + 4 + (2 if c["scaled"] else 0)
        per += 4 if c["gate"] == "full" else 0
        row = 8 + (8 if c["gate"] == "token" else 0)
        once += 4 * K + (4 * K if c["post"] else 0) + (6 * K if c["gate"] == "channel" else 0)
        return {"bytes": T * (K * per + row) + once, "flops": T * K * 20}
    if c["op"] == "router_balance":
        S = max(c["sequences"], 1)
        return {"bytes": T * (4 * c["E"] + 4 * c["topk"]) + 12 * S * c["E"], "flops": T * c["E"] * 6}
    if c["op"] == "router_backward":
        S = max(c["sequences"], 1)
        return {"bytes": T * (8 * c["E"] + 8 * c["topk"]) + 4 * S * c["E"], "flops": T * c["E"] * 12}
    K, k = c["K"], c["topk"]
    per = 1 + k + (k if c["routes_too"] else 0)
    return {"bytes": T * (2 * K * per + 4 * k * (2 if c["routes_too"] else 1)),
            "flops": T * K * k * (3 if c["routes_too"] else 2)}


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


def _mx8_values(q, scale):
    return q.double() * torch.exp2(scale.double() - 127).repeat_interleave(32, 1)


def _gate64(c, s):
    if s["gate"] is None:
        return torch.ones(1, 1, dtype=torch.float64, device=DEV)
    g = s["gate"].double()
    return torch.sigmoid(g) if c["act"] == "sigmoid" else g


def exact(case, seed):
    s, c = prepare(case, seed), case
    T = c["T"]
    if c["op"] == "sandwich_norm":
        x, K = s["x"].double(), c["K"]
        s1 = torch.ones(T, 1, dtype=torch.float64, device=DEV)
        n = x
        if c["post"]:
            s1 = torch.sqrt((x * x).sum(-1, keepdim=True) / K + EPS)
            n = x / s1 * s["g_post"].double()
        a = s["scale"].double() if c["scaled"] else 1.0
        h = a * s["res"].double() + _gate64(c, s) * n
        s2 = torch.sqrt((h * h).sum(-1, keepdim=True) / K + EPS)
        y = h / s2 * s["g_pre"].double()
        out = {"y": y, "h": h}
        if c["out8"]:
            out["q"], out["scale"] = _mx8_64(y, c["out8"])
        if c["train"]:
            out["rstd"] = torch.cat((1 / s1, 1 / s2), 1).t()
        if c["checkpoint8"]:
            out["x8"], out["x8_scale"] = _mx8_64(x, c["checkpoint8"])
            out["h8"], out["h8_scale"] = _mx8_64(h, c["checkpoint8"])
        return out
    if c["op"] == "sandwich_norm_backward":
        K = c["K"]
        if c["checkpoint8"]:
            x, h = _mx8_values(s["x"], s["sx"]), _mx8_values(s["h"], s["sh"])
        else:
            x, h = s["x"].double(), s["h"].double()
        r1, r2 = s["rstd"].double()[:, :, None]
        # the Jacobian of a norm with its factor kept: r (I - r^2 h h^T / K) diag(gamma)
        w = s["dy"].double() * s["g_pre"].double()
        dh = s["dh"].double() + r2 * w - r2 ** 3 / K * h * torch.linalg.vecdot(w, h)[:, None]
        out = {"pre_gamma": torch.einsum("tk,tk,tj->k", s["dy"].double(), h, r2)}
        out["residual"] = dh * (s["scale"].double() if c["scaled"] else 1.0)
        if c["scaled"]:
            out["residual_scale"] = torch.linalg.vecdot(dh, s["res"].double()).sum().reshape(1)
        gate = _gate64(c, s)
        dn = dh * gate
        n = x
        if c["post"]:
            gp = s["g_post"].double()
            n = x * r1 * gp
            out["post_gamma"] = torch.einsum("tk,tk,tj->k", dn, x, r1)
            out["x"] = r1 * gp * dn - r1 ** 3 / K * x * torch.linalg.vecdot(gp * dn, x)[:, None]
        else:
            out["x"] = dn
        if c["gate"]:
            d = dh * n * (gate * torch.sigmoid(-s["gate"].double()) if c["act"] == "sigmoid" else 1.0)
            out["gate"] = {"channel": lambda: d.sum(0, keepdim=True), "token": lambda: d.sum(1, keepdim=True),
                           "full": lambda: d}[c["gate"]]()
        return out
    if c["op"] == "combine_backward":
        K, k = c["K"], c["topk"]
        dy = s["dy"].double()
        o = s["routes"].double().view(T, k, K)
        out = {"weights": torch.stack([torch.linalg.vecdot(o[:, j], dy) for j in range(k)], 1)}
        if c["routes_too"]:
            out["routes"] = torch.stack([s["w"][:, j:j + 1].double() * dy for j in range(k)], 1).view(T * k, K)
        return out
    # the routers: sequence by sequence, gradients by differentiating the definition
    E, k = c["E"], c["topk"]
    x = s["logits"].double()
    ids = s["ids"].long()
    runs = [(0, T)]
    if s["offsets"] is not None:
        o = s["offsets"].tolist()
        runs = list(zip(o[:-1], o[1:]))
    if c["op"] == "router_backward":
        x.requires_grad_(True)
    score = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, -1)
    p = score / score.sum(-1, keepdim=True)
    lse2 = torch.logsumexp(x, -1) ** 2
    live = ids[:, 0] >= 0
    counts, prob, slope, losses = [], [], [], []
    zsum, tokens = torch.zeros((), dtype=torch.float64, device=DEV), 0
    for a, b in runs:
        rows = torch.nonzero(live[a:b]).flatten() + a
        n = rows.numel()
        cnt = torch.bincount(ids[rows].flatten(), minlength=E).double()
        counts.append(cnt.to(torch.int32))
        if n == 0:
            prob.append(torch.zeros(E, dtype=torch.float64, device=DEV))
            slope.append(torch.zeros(E, dtype=torch.float64, device=DEV))
            continue
        mean = p[rows].mean(0)
        frac = E * cnt / (k * n)
        prob.append(mean)
        slope.append(frac / n)
        losses.append((frac * mean).sum())
        zsum = zsum + lse2[rows].sum()
        tokens += n
    balance = sum(losses) / max(len(losses), 1) + torch.zeros((), dtype=torch.float64, device=DEV)
    z = zsum / max(tokens, 1)
    if c["op"] == "router_balance":
        rest = torch.tensor([float(tokens), float(len(losses))], dtype=torch.float64, device=DEV)
        return {"stats": torch.cat((torch.stack((balance, z)), rest)), "counts": torch.stack(counts),
                "prob": torch.stack(prob), "slope": torch.stack(slope)}
    w = score.gather(1, ids.clamp_min(0))
    if c["renormalise"]:
        w = w / w.sum(-1, keepdim=True)
    total = (w * c["scale"] * s["dw"].double())[live].sum()
    total = total + s["dloss"][0].double() * balance + s["dloss"][1].double() * z
    return {"logits": torch.autograd.grad(total, x)[0]}
