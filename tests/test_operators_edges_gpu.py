"""The operators around the layer where one wrong choice shows: sums that cancel,
memory and streams, lengths and limits at their ends."""
import numpy as np
import pytest
import torch

from oracle import operators_oracle as P
from test_operators_gpu import bits, call_linear, check_linear, f64, gen, make_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    from mxfp4_mixture_experts_gb300 import moe
    return moe


# ------------------------------------------------------------------ the adapters' inner products
def bf16_values(t):
    return t.double().numpy()


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("K,rank", [(64, 8), (192, 24), (128, 256), (1024, 40)])
@pytest.mark.parametrize("T", [1, 16, 17, 40, 130, 300])
def test_linear_adapter_whose_ranks_cancel(moe, T, K, rank, x8):
    """Zero weights, and adapters whose ranks come in pairs of almost equal inner products v with
    opposite signs in B: y is a small difference of large products. The tolerance has the output's
    rounding (2^-8 |y|), v's two bf16 values (2^-17 of the products' magnitudes) and the fp32 roundings
    of both sums (2^-23 of their magnitudes each: K / 16 steps, the adding of 8 warps and 8 parts and the
    factor for v, rank / 8 steps for y); one bf16 rounding of v (2^-9 of the products) is far outside."""
    d = make_linear(T, K, 136, rank, 3, x8, 1000 + T + K)
    g = gen(T)
    d["w"].zero_()
    a, b = d["adapter_a"], d["adapter_b"]
    a[:, 1::2] = (a[:, 0::2].float() * (1 + 2.0 ** -6 * torch.randn(3, rank // 2, K, generator=g))).bfloat16()
    b[:, :, 1::2] = -b[:, :, 0::2]
    d["adapter_ids"] = torch.randint(0, 3, (T,), generator=g, dtype=torch.int32)
    y = f64(call_linear(moe, d))
    n = (K / 16 + rank / 8 + 17) * 2.0 ** -23
    for t in range(T):
        j = int(d["adapter_ids"][t])
        A, B = bf16_values(a[j]), bf16_values(b[j])
        s, x = float(d["adapter_scale"][j]), d["x64"][t]
        v = A @ x * s
        ref = B @ v
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * (np.abs(B) @ np.abs(v)) \
            + n * (np.abs(B) @ (np.abs(A) @ np.abs(x) * s)) + 1e-37
        bad = np.abs(y[t] - ref) > tol
        assert not bad.any(), (t, y[t][bad][:4], ref[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("T", [2, 20, 300])
def test_linear_inner_product_beyond_bf16(moe, T):
    """An inner product between the largest bf16 and the largest fp32 value is finite, and so is y."""
    d = make_linear(T, 64, 16, 8, 1, False, 5, 0)
    d["w"].zero_()
    d["x"].fill_(1.0)
    d["adapter_a"].zero_()
    d["adapter_a"][0, 0, 0] = 1.0
    d["adapter_b"].fill_(0.5)
    d["adapter_scale"].fill_(3.4e38)
    y = f64(call_linear(moe, d))
    assert np.all(np.abs(y - 1.7e38) <= 1.7e38 * 2.0 ** -8)


# ------------------------------------------------------------------ memory of calls on another stream
def late_writer(shapes, dtype=torch.uint8):
    """Blocks of these sizes that the current stream will still write to, 20 ms from now, although they are
    free for its next allocations."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    tmp = [torch.empty(n, dtype=dtype, device="cuda") for n in shapes]
    torch.cuda._sleep(40_000_000)
    for t in tmp:
        t.fill_(0xFF)


def stream_calls(moe):
    """name -> (call with a stream, bytes of its outputs and scratch); all larger than the allocator's pool of
    small blocks, inputs long ready."""
    g = gen(77)
    x = torch.randn(1024, 2048, generator=g).bfloat16().cuda()
    gamma = torch.ones(2048).bfloat16().cuda()
    logits = torch.randn(70_000, 64, generator=g).cuda()
    d = {k: v.cuda() for k, v in make_linear(1200, 1024, 2048, 16, 3, True, 78).items() if k != "x64"}
    lin = lambda st: moe.linear(d["x"], d["w"], d["s"], d["x_scale"], d["adapter_ids"], d["adapter_a"],
                                d["adapter_b"], d["adapter_scale"], stream=st)
    return {
        "add_rmsnorm": (lambda st: moe.add_rmsnorm(x, gamma, x, out8="ocp", stream=st)[:3],
                        [1024 * 2048 * 2] * 2 + [1024 * 2048]),
        "router_scored": (lambda st: moe.router_scored(logits, 8, stream=st), [70_000 * 8 * 4] * 2),
        "linear": (lin, [1200 * 2048 * 2, moe.linear_workspace_size(1200, 1024, 2048, 16, True)]),
    }


@pytest.mark.parametrize("op", ["add_rmsnorm", "router_scored", "linear"])
def test_call_on_another_stream_does_not_share_memory_with_queued_work(moe, op):
    call, sizes = stream_calls(moe)[op]
    as_bytes = lambda r: [t.view(torch.uint8).clone() for t in (r if isinstance(r, tuple) else (r,))]
    want = as_bytes(call(None))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    late_writer(sizes)
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(want, as_bytes(got)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("op", ["add_rmsnorm", "router_scored", "linear"])
def test_call_on_another_stream_allocates_there(moe, monkeypatch, op):
    call, sizes = stream_calls(moe)[op]
    side = torch.cuda.Stream()
    seen = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (seen.append(torch.cuda.current_stream()), empty(*a, **k))[1])
    call(side)
    assert len(seen) >= len(sizes) and all(s == side for s in seen)
    torch.cuda.synchronize()


def test_outputs_of_another_stream_outlive_their_reader(moe):
    """An output that the current stream still reads when it is dropped is not handed to the side stream's next call."""
    g = gen(79)
    x, y = (torch.randn(1024, 2048, generator=g).bfloat16().cuda() for _ in range(2))
    gamma = torch.ones(2048).bfloat16().cuda()
    want = moe.add_rmsnorm(x, gamma)[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = moe.add_rmsnorm(x, gamma, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(40_000_000)
    copy = a.clone()
    del a
    moe.add_rmsnorm(y, gamma, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


def layer_calls(moe):
    """The layer's own calls with a stream, by name, outputs as a tuple."""
    g = gen(80)
    u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.uint8).cuda()
    T, K, I, E = 300, 256, 128, 8
    h = torch.randn(T, K, generator=g).bfloat16().cuda()
    logits = torch.randn(T, E, generator=g).cuda()
    ids, w = moe.router(logits, 2)
    w13, s13, w2, s2 = u8(0, 256, E, 2 * I, K // 2), u8(118, 124, E, 2 * I, K // 32), \
        u8(0, 256, E, K, I // 2), u8(118, 124, E, K, I // 32)
    b13, b2 = torch.zeros(E, 2 * I).cuda(), torch.zeros(E, K).cuda()
    lay = dict(
        route=lambda st: moe.route(ids, E, stream=st),
        route_many=lambda st: moe.route(ids, E, stream=st, many_ctas=True),
        router=lambda st: moe.router(logits, 2, stream=st),
        router_grouped=lambda st: moe.router_grouped(logits, 2, n_group=2, topk_group=1, stream=st),
        encode=lambda st: moe.encode(h, stream=st),
        dequant=lambda st: (moe.dequant(w2[0], s2[0], stream=st),),
        forward=lambda st: (moe.forward(h, ids, w, w13, s13, w2, s2, stream=st),),
        forward_decode=lambda st: (moe.forward(h[:8], ids[:8], w[:8], w13, s13, w2, s2, stream=st),),
        forward_window=lambda st: (moe.forward_window(h, ids, w, w13, s13, w2, s2, stream=st),),
        forward_oai=lambda st: (moe.forward_oai(h, ids, w, w13, s13, b13, w2, s2, b2, stream=st),),
    )
    return lay


@pytest.mark.parametrize("op", ["route", "route_many", "router", "router_grouped", "encode", "dequant", "forward",
                                "forward_decode", "forward_window", "forward_oai"])
def test_layer_call_on_another_stream_allocates_and_zeroes_there(moe, monkeypatch, op):
    call = layer_calls(moe)[op]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    seen = []
    empty, zeros = torch.empty, torch.zeros
    spy = lambda f: lambda *a, **k: (seen.append(torch.cuda.current_stream()), f(*a, **k))[1]
    monkeypatch.setattr(torch, "empty", spy(empty))
    monkeypatch.setattr(torch, "zeros", spy(zeros))
    torch.cuda._sleep(40_000_000)     # the current stream is busy, the call's is not
    got = call(side)
    side.synchronize()
    assert seen and all(s == side for s in seen)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------ threads
FIRST_CALLS = """
import sys, threading
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
from mxfp4_mixture_experts_gb300 import moe
from test_operators_gpu import make_linear
d = {{k: v.cuda() for k, v in make_linear(32, 6144, 4096, 16, 5, False, 3).items() if k != "x64"}}
torch.cuda.synchronize()
moe.lib()
n = 12
start, out, errors = threading.Barrier(n), [None] * n, []
def first(i):
    try:
        st = torch.cuda.Stream()
        start.wait()
        out[i] = moe.linear(d["x"], d["w"], d["s"], None, d["adapter_ids"], d["adapter_a"], d["adapter_b"],
                            d["adapter_scale"], stream=st)
        st.synchronize()
    except Exception as e:
        errors.append(e)
threads = [threading.Thread(target=first, args=(i,)) for i in range(n)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not errors, errors
again = moe.linear(d["x"], d["w"], d["s"], None, d["adapter_ids"], d["adapter_a"], d["adapter_b"], d["adapter_scale"])
assert all(torch.equal(o, again) for o in out)
print("equal")
"""


def test_first_calls_of_several_threads_agree(moe):
    """The first projections of a process, from twelve threads at once, choose the same tiles: the same bits."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=root)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------------------ long calls
def test_linear_call_of_seconds_is_not_reported_as_a_failure(moe):
    """The waits' bound of 0.2 s is one for each wait, not for the call: a projection of a second
    (every token another adapter of 256 ranks, as many columns to a tile as there can be)."""
    T, K, N, L, rank = 131_072, 64, 16_384, 256, 256
    g = torch.Generator(device="cuda").manual_seed(9)
    rn = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    x, a, b = rn(T, K), rn(L, rank, K), rn(L, N, rank)
    w = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.full((N, K // 32), 122, dtype=torch.uint8, device="cuda")
    ids = (torch.arange(T, device="cuda") * 37 % L).to(torch.int32)
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    status = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    start, end = torch.cuda.Event(True), torch.cuda.Event(True)
    start.record()
    moe.linear(x, w, s, adapter_ids=ids, adapter_a=a, adapter_b=b, out=out, status=status)
    end.record()
    torch.cuda.synchronize()
    print(f"{start.elapsed_time(end):.0f} ms")
    assert start.elapsed_time(end) > 600     # (else this test shows nothing)
    assert status.tolist() == [0, 0, 0, 0]
    for t in (0, 1, 255, 256, 100_003, T - 1):
        j = int(ids[t])
        ref, mag, low = P.linear(f64(x[t:t + 1]), w.cpu().numpy(), s.cpu().numpy(), [0], bits(a[j:j + 1]),
                                 bits(b[j:j + 1]))
        tol = 2.0 ** -8 * np.abs(ref) + (K / 16 + rank / 8 + 17) * 2.0 ** -23 * (mag + 8 * low) + 2.0 ** -17 * low
        assert np.all(np.abs(f64(out[t:t + 1]) - ref) <= tol)
    del x, a, b, out
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ the most rows that a call can name
def test_add_rmsnorm_of_the_most_rows(moe):
    """2^31 - 1 rows (137 GB, in place): the row after a CTA's last one is past 2^31."""
    T, K = 2 ** 31 - 1, 32
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 150e9:
        pytest.skip("needs 150 GB of free device memory")
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").fill_(1.0)
    rows = torch.tensor([0, 1215, 1216, 2 ** 30, 2 ** 31 - 1217, 2 ** 31 - 1216, T - 2, T - 1], device="cuda")
    vals = torch.arange(len(rows), device="cuda").float()[:, None].expand(-1, K).bfloat16() + 2
    x[rows] = vals
    none, h, _, _ = moe.add_rmsnorm(x, torch.ones(K, device="cuda").bfloat16(), x, bf16=False, residual_out=x)
    torch.cuda.synchronize()
    assert none is None and h is x
    assert torch.equal(x[rows], 2 * vals)
    for r in (2, 2 ** 29 + 1, 2 ** 31 - 5000):
        assert (x[r:r + 1000] == 2).all()
    del x, h
    torch.cuda.empty_cache()


def test_router_scored_of_the_most_rows(moe):
    """2^31 - 1 rows of one expert (26 GB)."""
    T = 2 ** 31 - 1
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB of free device memory")
    x = torch.zeros(T, 1, device="cuda")
    x[-2] = float("nan")
    ids = torch.full((T, 1), 7, dtype=torch.int32, device="cuda")
    ids, w = moe.router_scored(x, 1, "softmax", topk_ids=ids)
    torch.cuda.synchronize()
    assert int(ids[-2]) == -1 and float(w[-2]) == 0.0
    assert int((ids == 0).sum()) == T - 1 and int((w == 1).sum()) == T - 1
    del x, ids, w
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ waits that give up
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("rank", [0, 16])
@pytest.mark.parametrize("T,cta", [(40, 0), (40, 3), (700, 1)])
def test_linear_missing_copy_is_reported_and_the_next_call_is_right(moe, T, cta, rank, x8):
    """A copy that never comes (K split over a cluster; one pair a tile): the call ends within its bounds and
    says so, and the same workspace serves the next one. No GPU fault and no endless wait is involved."""
    K, N = 2048, 1032
    d = {k: v.cuda() for k, v in make_linear(T, K, N, rank, 5, x8, 60 + T).items() if k != "x64"}
    x, w, s, xs = d.pop("x"), d.pop("w"), d.pop("s"), d.pop("x_scale", None)
    want = moe.linear(x, w, s, xs, **d)
    ws = torch.empty(max(moe.linear_workspace_size(T, K, N, rank, x8), 1), dtype=torch.uint8, device="cuda")
    status = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    start, end = torch.cuda.Event(True), torch.cuda.Event(True)
    moe.lib().mxfp4_moe_test_skip_linear_copy(cta)
    try:
        start.record()
        moe.linear(x, w, s, xs, workspace=ws, status=status, **d)
        end.record()
        torch.cuda.synchronize()
    finally:
        moe.lib().mxfp4_moe_test_skip_linear_copy(-1)
    beyond = int((d["adapter_ids"] >= 5).sum()) if rank else 0
    assert status[:3].tolist() == [beyond, 0, 1] and 1 <= int(status[3]) <= 152
    assert start.elapsed_time(end) < 10_000
    y = moe.linear(x, w, s, xs, workspace=ws, status=status, **d)
    torch.cuda.synchronize()
    assert status.tolist() == [beyond, 0, 0, 0] and torch.equal(y, want)


# ------------------------------------------------------------------ limits of the projection's sizes
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("T", [5, 24, 300])
def test_linear_longest_rows_and_most_adapters(moe, T, x8):
    """K = 16384 and 1024 adapters, a token each, the last ones among them."""
    d = make_linear(T, 16384, 136, 8, 1024, x8, 2000 + T)
    d["adapter_ids"] = (1023 - torch.arange(T) * 3 % 1024).to(torch.int32)
    check_linear(moe, d)


@pytest.mark.parametrize("T", [3, 40, 300])
def test_linear_smallest_and_largest_scales_are_exact(moe, T):
    """Weights and MXFP8 rows whose scales make them bf16's subnormal numbers (rows from scale byte 3 on, below
    which a code's last bits are under bf16's smallest step), against factors that bring y back into range."""
    for low in ("x", "w"):
        d = make_linear(T, 256, 136, 0, 0, True, 31)
        sx = torch.randint(*((3, 8) if low == "x" else (228, 232)), d["x_scale"].shape, generator=gen(1), dtype=torch.uint8)
        sw = torch.randint(*((0, 4) if low == "w" else (228, 232)), d["s"].shape, generator=gen(2), dtype=torch.uint8)
        q = d["x"].double().numpy()
        d["x_scale"], d["s"] = sx, sw
        d["x64"] = q * np.repeat(np.exp2(sx.numpy().astype(np.float64) - 127), 32, 1)
        check_linear(moe, d)
