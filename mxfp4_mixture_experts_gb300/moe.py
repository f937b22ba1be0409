"""ctypes binding of libmxfp4_moe.so (C ABI: include/mxfp4_moe.h).

Argument marshalling only: every entry point takes PyTorch CUDA tensors,
checks dtype / shape / device, and passes raw device pointers plus the current
CUDA stream to the library. All computation happens in the library's kernels;
there is no fallback: if the library is missing or a call fails, an exception
is raised.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxfp4_moe.so")

OK, ERR_ARG, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE = range(7)

_lib = None


class MoEError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} (code {code})")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with mxfp4_mixture_experts_gb300.build.build()")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.mxfp4_moe_workspace_size.argtypes = [i32] * 5
    L.mxfp4_moe_workspace_size.restype = sz
    L.mxfp4_moe_workspace_zero_bytes.argtypes = []
    L.mxfp4_moe_workspace_zero_bytes.restype = sz
    L.mxfp4_moe_route.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp]
    L.mxfp4_moe_route.restype = i32
    L.mxfp4_moe_route_workspace_size.argtypes = [i32, i32, i32]
    L.mxfp4_moe_route_workspace_size.restype = sz
    L.mxfp4_moe_route_ws.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    L.mxfp4_moe_route_ws.restype = i32
    L.mxfp4_moe_forward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                    vp, vp, vp, sz, i32, vp]
    L.mxfp4_moe_forward.restype = i32
    L.mxfp4_moe_forward_oai.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                        i32, vp, vp, vp, sz, i32, vp]
    L.mxfp4_moe_forward_oai.restype = i32
    L.mxfp4_moe_router.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp]
    L.mxfp4_moe_router.restype = i32
    L.mxfp4_moe_router_grouped.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp, vp]
    L.mxfp4_moe_router_grouped.restype = i32
    L.mxfp4_moe_forward_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32,
                                           i32, i32, vp, vp, vp, sz, i32, vp]
    L.mxfp4_moe_forward_window.restype = i32
    L.mxfp4_moe_encode.argtypes = [vp, i32, i32, i32, vp, vp, vp]
    L.mxfp4_moe_encode.restype = i32
    L.mxfp4_moe_dequant.argtypes = [vp, vp, i32, i32, vp, vp]
    L.mxfp4_moe_dequant.restype = i32
    L.mxfp4_moe_dequant_form.argtypes = [vp, vp, i32, i32, i32, vp, vp]
    L.mxfp4_moe_dequant_form.restype = i32
    f32 = ctypes.c_float
    L.mxfp4_moe_add_rmsnorm.argtypes = [vp, vp, vp, i32, i32, f32, i32, vp, vp, vp, vp, vp]
    L.mxfp4_moe_add_rmsnorm.restype = i32
    L.mxfp4_moe_router_scored.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, f32,
                                          vp, vp, vp]
    L.mxfp4_moe_router_scored.restype = i32
    L.mxfp4_moe_sandwich_norm.argtypes = [vp] * 5 + [i32, i32, vp, i32, i32, f32, i32, i32] + [vp] * 10
    L.mxfp4_moe_sandwich_norm.restype = i32
    L.mxfp4_moe_sandwich_norm_backward_workspace_size.argtypes = [i32, i32]
    L.mxfp4_moe_sandwich_norm_backward_workspace_size.restype = sz
    L.mxfp4_moe_sandwich_norm_backward.argtypes = [vp] * 10 + [i32, i32, vp, vp, i32, i32] + \
        [vp] * 7 + [sz, vp]
    L.mxfp4_moe_sandwich_norm_backward.restype = i32
    L.mxfp4_moe_router_balance_workspace_size.argtypes = [i32] * 3
    L.mxfp4_moe_router_balance_workspace_size.restype = sz
    L.mxfp4_moe_router_balance.argtypes = [vp, vp, i32, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp,
                                           sz, vp]
    L.mxfp4_moe_router_balance.restype = i32
    L.mxfp4_moe_router_backward.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, f32, vp, vp, vp, vp,
                                            i32, vp, vp]
    L.mxfp4_moe_router_backward.restype = i32
    L.mxfp4_moe_combine_backward.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp]
    L.mxfp4_moe_combine_backward.restype = i32
    L.mxfp4_moe_linear_workspace_size.argtypes = [i32] * 5
    L.mxfp4_moe_linear_workspace_size.restype = sz
    L.mxfp4_moe_linear.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, i32, i32,
                                   vp, vp, vp, sz, vp]
    L.mxfp4_moe_linear.restype = i32
    L.mxfp4_moe_test_skip_grid_arrival.argtypes = [i32]
    L.mxfp4_moe_test_skip_grid_arrival.restype = None
    L.mxfp4_moe_test_skip_linear_copy.argtypes = [i32]
    L.mxfp4_moe_test_skip_linear_copy.restype = None
    L.mxfp4_moe_test_decode_form.argtypes = [i32] * 6
    L.mxfp4_moe_test_decode_form.restype = i32
    L.mxfp4_moe_set_phase_events.argtypes = [vp, i32]
    L.mxfp4_moe_set_phase_events.restype = None
    L.mxfp4_moe_strerror.argtypes = [i32]
    L.mxfp4_moe_strerror.restype = ctypes.c_char_p
    L.mxfp4_moe_version.argtypes = []
    L.mxfp4_moe_version.restype = i32
    _lib = L
    return L


def decode_form(T: int, K: int, I: int, E: int, topk: int, max_smem: int = 232448) -> int:
    """Warps per CTA of the decode form a call of this shape and T runs (7: seven
    consumer warps and a producer), 0 when none fits, -1 for shapes the decode
    path does not take. Host only (227 KB of shared memory per block by default)."""
    return lib().mxfp4_moe_test_decode_form(T, K, I, E, topk, max_smem)


def strerror(code: int) -> str:
    return lib().mxfp4_moe_strerror(int(code)).decode()


def version() -> int:
    return lib().mxfp4_moe_version()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _addr(t: Optional[torch.Tensor]):
    """The device address as an int (what ctypes makes of a declared pointer argument anyway)."""
    return None if t is None else t.data_ptr()


def _raw_stream(stream) -> int:
    """The cudaStream_t of ``stream``, or of the current stream, without the Stream object that
    torch.cuda.current_stream builds (0.2 against 2.8 us a call)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An uninitialised tensor for a call on ``stream``, from that stream's own memory: what other
    streams have freed may still be in use by their queued work. Nor is its memory handed out again
    before the current stream, where the caller may use it, has passed the point that drops it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _zeros(shape, dtype, device, stream) -> torch.Tensor:
    """``_empty``, zeroed on ``stream``."""
    if stream is None:
        return torch.zeros(shape, dtype=dtype, device=device)
    t = _empty(shape, dtype, device, stream)
    with torch.cuda.stream(stream):
        return t.zero_()


def _need(t: torch.Tensor, name: str, dtype, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def workspace_size(T: int, K: int, I: int, E: int, topk: int) -> int:
    return int(lib().mxfp4_moe_workspace_size(T, K, I, E, topk))


def workspace_zero_bytes() -> int:
    """Bytes at the start of a workspace that must be zero before first use
    (every call leaves them zero)."""
    return int(lib().mxfp4_moe_workspace_zero_bytes())


def new_workspace(T: int, K: int, I: int, E: int, topk: int, device="cuda",
                  stream=None) -> torch.Tensor:
    """A zero-filled workspace (the library requires zeros before first use), zeroed on ``stream``
    (the current one by default)."""
    n = workspace_size(T, K, I, E, topk)
    if n == 0:
        raise ValueError("unsupported sizes")
    return _zeros(n, torch.uint8, device, stream)


def route(topk_ids: torch.Tensor, E: int, stream=None, many_ctas: bool = False):
    """Stable counting sort of routes by expert -> (count[E], offset[E+1],
    route_list[T*k], status[4]), all int32 CUDA tensors. many_ctas takes
    mxfp4_moe_route_ws (the prefill path's sort, over many CTAs from 8192
    routes on) with scratch allocated here."""
    _need(topk_ids, "topk_ids", torch.int32, 2)
    T, k = topk_ids.shape
    dev = topk_ids.device
    count = _empty(E, torch.int32, dev, stream)
    offset = _empty(E + 1, torch.int32, dev, stream)
    lst = _empty(max(T * k, 1), torch.int32, dev, stream)
    status = _zeros(4, torch.int32, dev, stream)
    if many_ctas:
        n = int(lib().mxfp4_moe_route_workspace_size(T, k, E))
        ws = _empty(max(n, 16), torch.uint8, dev, stream)
        rc = lib().mxfp4_moe_route_ws(_ptr(topk_ids), T, k, E, _ptr(count), _ptr(offset),
                                      _ptr(lst), _ptr(status), _ptr(ws), n, _stream(stream))
        if rc:
            raise MoEError(rc, "mxfp4_moe_route_ws")
    else:
        rc = lib().mxfp4_moe_route(_ptr(topk_ids), T, k, E, _ptr(count), _ptr(offset),
                                   _ptr(lst), _ptr(status), _stream(stream))
        if rc:
            raise MoEError(rc, "mxfp4_moe_route")
    return count, offset, lst[:T * k], status


def forward(hidden: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
            w13: torch.Tensor, s13: torch.Tensor, w2: torch.Tensor, s2: torch.Tensor,
            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
            status: Optional[torch.Tensor] = None, path: int = 0, stream=None) -> torch.Tensor:
    """y[T, K] bf16 = sum_j w_tj * W2[e] (silu(W_gate[e] x_t) * (W_up[e] x_t))."""
    _need(hidden, "hidden", torch.bfloat16, 2)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    _need(topk_weights, "topk_weights", torch.float32, 2)
    for n, t in (("w13", w13), ("s13", s13), ("w2", w2), ("s2", s2)):
        _need(t, n, torch.uint8, 3)
    T, K = hidden.shape
    E, twoI, _ = w13.shape
    I = twoI // 2
    k = topk_ids.shape[1]
    if tuple(topk_ids.shape) != (T, k) or tuple(topk_weights.shape) != (T, k):
        raise ValueError("topk_ids / topk_weights must be [T, topk]")
    if tuple(w13.shape) != (E, 2 * I, K // 2) or tuple(s13.shape) != (E, 2 * I, K // 32):
        raise ValueError("w13 / s13 shapes must be [E, 2I, K/2] / [E, 2I, K/32]")
    if tuple(w2.shape) != (E, K, I // 2) or tuple(s2.shape) != (E, K, I // 32):
        raise ValueError("w2 / s2 shapes must be [E, K, I/2] / [E, K, I/32]")
    if out is None:
        out = _empty((T, K), torch.bfloat16, hidden.device, stream)
    else:
        _need(out, "out", torch.bfloat16, 2)
    if workspace is None:
        workspace = new_workspace(T, K, I, E, k, hidden.device, stream)
    rc = lib().mxfp4_moe_forward(
        _ptr(hidden), _ptr(topk_ids), _ptr(topk_weights), _ptr(w13), _ptr(s13), _ptr(w2),
        _ptr(s2), T, K, I, E, k, _ptr(out), _ptr(status), _ptr(workspace),
        workspace.numel() * workspace.element_size(), path, _stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_forward")
    return out


def forward_window(hidden: torch.Tensor, topk_ids: torch.Tensor,
                   topk_weights: Optional[torch.Tensor], w13: torch.Tensor, s13: torch.Tensor,
                   w2: torch.Tensor, s2: torch.Tensor, expert_base: int = 0,
                   per_route: bool = False, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                   path: int = 0, stream=None) -> torch.Tensor:
    """The layer over the experts expert_base .. expert_base + E - 1 held by
    w13/s13/w2/s2 (other ids skipped): y [T, K] of the window's routes, or with
    per_route each route's unweighted w2 output [T * topk, K]."""
    _need(hidden, "hidden", torch.bfloat16, 2)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, 2)
    elif not per_route:
        raise ValueError("topk_weights are needed unless per_route")
    for n, t in (("w13", w13), ("s13", s13), ("w2", w2), ("s2", s2)):
        _need(t, n, torch.uint8, 3)
    T, K = hidden.shape
    E, twoI, _ = w13.shape
    I = twoI // 2
    k = topk_ids.shape[1]
    rows = T * k if per_route else T
    if out is None:
        out = _empty((rows, K), torch.bfloat16, hidden.device, stream)
    else:
        _need(out, "out", torch.bfloat16, 2)
        if tuple(out.shape) != (rows, K):
            raise ValueError(f"out must be [{rows}, {K}]")
    if workspace is None:
        workspace = new_workspace(T, K, I, E, k, hidden.device, stream)
    rc = lib().mxfp4_moe_forward_window(
        _ptr(hidden), _ptr(topk_ids), _ptr(topk_weights), _ptr(w13), _ptr(s13), _ptr(w2),
        _ptr(s2), T, K, I, E, k, int(expert_base), int(bool(per_route)), _ptr(out), _ptr(status),
        _ptr(workspace), workspace.numel() * workspace.element_size(), path, _stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_forward_window")
    return out


def forward_oai(hidden: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                w13: torch.Tensor, s13: torch.Tensor, b13: torch.Tensor,
                w2: torch.Tensor, s2: torch.Tensor, b2: torch.Tensor,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None, path: int = 0, stream=None) -> torch.Tensor:
    """The gpt-oss form: w13 rows interleaved (row 2i gate i, row 2i + 1 up i),
    f32 biases b13 [E, 2I] (same row order) and b2 [E, K], SwiGLU-OAI;
    y[T, K] bf16 = sum_j w_tj * (W2[e] h + b2[e]). Paths as forward()."""
    _need(hidden, "hidden", torch.bfloat16, 2)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    _need(topk_weights, "topk_weights", torch.float32, 2)
    for n, t in (("w13", w13), ("s13", s13), ("w2", w2), ("s2", s2)):
        _need(t, n, torch.uint8, 3)
    _need(b13, "b13", torch.float32, 2)
    _need(b2, "b2", torch.float32, 2)
    T, K = hidden.shape
    E, twoI, _ = w13.shape
    I = twoI // 2
    k = topk_ids.shape[1]
    if tuple(topk_ids.shape) != (T, k) or tuple(topk_weights.shape) != (T, k):
        raise ValueError("topk_ids / topk_weights must be [T, topk]")
    if tuple(w13.shape) != (E, 2 * I, K // 2) or tuple(s13.shape) != (E, 2 * I, K // 32):
        raise ValueError("w13 / s13 shapes must be [E, 2I, K/2] / [E, 2I, K/32]")
    if tuple(w2.shape) != (E, K, I // 2) or tuple(s2.shape) != (E, K, I // 32):
        raise ValueError("w2 / s2 shapes must be [E, K, I/2] / [E, K, I/32]")
    if tuple(b13.shape) != (E, 2 * I) or tuple(b2.shape) != (E, K):
        raise ValueError("b13 / b2 shapes must be [E, 2I] / [E, K]")
    if out is None:
        out = _empty((T, K), torch.bfloat16, hidden.device, stream)
    else:
        _need(out, "out", torch.bfloat16, 2)
    if workspace is None:
        workspace = new_workspace(T, K, I, E, k, hidden.device, stream)
    rc = lib().mxfp4_moe_forward_oai(
        _ptr(hidden), _ptr(topk_ids), _ptr(topk_weights), _ptr(w13), _ptr(s13), _ptr(b13),
        _ptr(w2), _ptr(s2), _ptr(b2), T, K, I, E, k, _ptr(out), _ptr(status), _ptr(workspace),
        workspace.numel() * workspace.element_size(), path, _stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_forward_oai")
    return out


SCORING = {"softmax_topk": 0, "sigmoid_renorm": 1}


def _router_args(logits, topk, scoring, bias, topk_ids, topk_weights, stream):
    _need(logits, "logits", torch.float32, 2)
    T, E = logits.shape
    if bias is not None:
        _need(bias, "bias", torch.float32, 1)
        if bias.shape[0] != E:
            raise ValueError("bias must be [E]")
    if scoring not in SCORING:
        raise ValueError(f"scoring must be one of {sorted(SCORING)}")
    if topk_ids is None:
        topk_ids = _empty((T, topk), torch.int32, logits.device, stream)
    if topk_weights is None:
        topk_weights = _empty((T, topk), torch.float32, logits.device, stream)
    return T, E, topk_ids, topk_weights


def router(logits: torch.Tensor, topk: int, scoring: str = "softmax_topk",
           bias: Optional[torch.Tensor] = None, topk_ids: Optional[torch.Tensor] = None,
           topk_weights: Optional[torch.Tensor] = None, stream=None):
    """Top-k experts of fp32 logits [T, E] (+ bias [E]) and their weights:
    int32 [T, k] ids (descending x = logit + bias, ties to the lower index)
    and fp32 [T, k] weights (softmax over the chosen, or renormalised sigmoid)."""
    T, E, topk_ids, topk_weights = _router_args(logits, topk, scoring, bias, topk_ids,
                                                topk_weights, stream)
    rc = lib().mxfp4_moe_router(_ptr(logits), _ptr(bias), T, E, topk, SCORING[scoring],
                                _ptr(topk_ids), _ptr(topk_weights), _stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_router")
    return topk_ids, topk_weights


def router_grouped(logits: torch.Tensor, topk: int, scoring: str = "sigmoid_renorm",
                   bias: Optional[torch.Tensor] = None, n_group: int = 1, topk_group: int = 1,
                   bias_in_weights: bool = True, topk_ids: Optional[torch.Tensor] = None,
                   topk_weights: Optional[torch.Tensor] = None, stream=None):
    """``router`` with grouped top-k (n_group groups of consecutive experts
    scored by their largest x; the experts of the topk_group best groups stay
    eligible) and, with bias_in_weights=False, a bias that steers the choice
    only (weights from the unbiased logits)."""
    T, E, topk_ids, topk_weights = _router_args(logits, topk, scoring, bias, topk_ids,
                                                topk_weights, stream)
    rc = lib().mxfp4_moe_router_grouped(_ptr(logits), _ptr(bias), T, E, topk, SCORING[scoring],
                                        n_group, topk_group, int(bool(bias_in_weights)),
                                        _ptr(topk_ids), _ptr(topk_weights), _stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_router_grouped")
    return topk_ids, topk_weights


RULES = {"ocp": 0, "quark": 1}


def encode(x: torch.Tensor, rule: str = "ocp", stream=None):
    """bf16 [rows, cols] -> (packed uint8 [rows, cols/2], E8M0 scales uint8
    [rows, cols/32]); rule "ocp" (floor(log2 amax) - 2) or "quark" (raised by
    one when amax / 2^X >= 7)."""
    _need(x, "x", torch.bfloat16, 2)
    if rule not in RULES:
        raise ValueError(f"rule must be one of {sorted(RULES)}")
    rows, cols = x.shape
    packed = _empty((rows, cols // 2), torch.uint8, x.device, stream)
    scale = _empty((rows, cols // 32), torch.uint8, x.device, stream)
    rc = lib().mxfp4_moe_encode(_ptr(x), rows, cols, RULES[rule], _ptr(packed), _ptr(scale),
                                _stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_encode")
    return packed, scale


DEQUANT_FORMS = {"decode": 1, "prefill": 2}


def dequant(packed: torch.Tensor, scale: torch.Tensor, form: str = "decode",
            stream=None) -> torch.Tensor:
    """Packed rows [N, C/2] + scales [N, C/32] -> bf16 [N, C], through the
    weight decode of the decode kernels (form "decode") or of the prefill
    GEMM (form "prefill")."""
    _need(packed, "packed", torch.uint8, 2)
    _need(scale, "scale", torch.uint8, 2)
    if form not in DEQUANT_FORMS:
        raise ValueError(f"form must be one of {sorted(DEQUANT_FORMS)}")
    N, half = packed.shape
    C = 2 * half
    if tuple(scale.shape) != (N, C // 32):
        raise ValueError("scale must be [rows, cols/32]")
    out = _empty((N, C), torch.bfloat16, packed.device, stream)
    rc = lib().mxfp4_moe_dequant_form(_ptr(packed), _ptr(scale), N, C, DEQUANT_FORMS[form],
                                      _ptr(out), _stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_dequant_form")
    return out


MX8_RULES = {"ocp": 0, "nosat": 1}


def add_rmsnorm(x: torch.Tensor, gamma: torch.Tensor, residual: Optional[torch.Tensor] = None,
                eps: float = 1e-5, out8: Optional[str] = None, bf16: bool = True,
                residual_out: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None):
    """h = x + residual, y = h * rsqrt(mean(h^2) + eps) * gamma for bf16 rows [T, K].

    Returns (y bf16 or None, bf16(h), q8, s8): y unless bf16 is False; the new
    residual stream (x itself when there is no residual; residual_out may be x
    or residual); with out8 "ocp" or "nosat" y's MXFP8 form, E4M3 [T, K] and
    E8M0 bytes [T, K/32] (the exponent floor(log2 amax) - 8, under "nosat"
    raised by one where the block would saturate), else None."""
    _need(x, "x", torch.bfloat16, 2)
    _need(gamma, "gamma", torch.bfloat16, 1)
    shape = x.shape
    T, K = shape
    if gamma.shape[0] != K:
        raise ValueError("gamma must be [K]")
    if out8 is not None and out8 not in MX8_RULES:
        raise ValueError(f"out8 must be None or one of {sorted(MX8_RULES)}")
    dev = x.device
    if residual is not None:
        _need(residual, "residual", torch.bfloat16, 2)
        if residual.shape != shape:
            raise ValueError("residual must be [T, K]")
    if residual_out is not None:
        _need(residual_out, "residual_out", torch.bfloat16, 2)
        if residual_out.shape != shape:
            raise ValueError("residual_out must be [T, K]")
    elif residual is not None:
        residual_out = _empty(shape, torch.bfloat16, dev, stream)
    if out is not None:
        if not bf16:
            raise ValueError("out is not written when bf16 is False")
        _need(out, "out", torch.bfloat16, 2)
        if out.shape != shape:
            raise ValueError("out must be [T, K]")
    elif bf16:
        out = _empty(shape, torch.bfloat16, dev, stream)
    q = s = None
    if out8 is not None:
        q = _empty(shape, torch.float8_e4m3fn, dev, stream)
        s = _empty((T, K // 32), torch.uint8, dev, stream)
    rc = lib().mxfp4_moe_add_rmsnorm(_addr(x), _addr(residual), _addr(gamma), T, K, eps,
                                     MX8_RULES[out8 or "ocp"], _addr(residual_out), _addr(out),
                                     _addr(q), _addr(s), _raw_stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_add_rmsnorm")
    return out, (x if residual_out is None else residual_out), q, s


SCORES = {"softmax": 0, "sigmoid": 1}


def router_scored(logits: torch.Tensor, topk: int, scoring: str = "sigmoid",
                  bias: Optional[torch.Tensor] = None, n_group: int = 1, topk_group: int = 1,
                  group_top: int = 2, renormalise: bool = True, route_scale: float = 1.0,
                  topk_ids: Optional[torch.Tensor] = None,
                  topk_weights: Optional[torch.Tensor] = None, stream=None):
    """Top-k experts by score: s = sigmoid(logits) or softmax over all experts
    of fp32 logits [T, E], chosen by s + bias [E] (ties to the lower index)
    among the topk_group groups with the largest sums of their group_top best;
    weights from s alone, renormalised over the chosen or not, times
    route_scale. Experts with a NaN or -inf logit are never chosen; a slot with
    none left gets id -1 and weight 0. Returns int32 ids and fp32 weights [T, k]."""
    _need(logits, "logits", torch.float32, 2)
    T, E = logits.shape
    if scoring not in SCORES:
        raise ValueError(f"scoring must be one of {sorted(SCORES)}")
    if bias is not None:
        _need(bias, "bias", torch.float32, 1)
        if bias.shape[0] != E:
            raise ValueError("bias must be [E]")
    if topk_ids is None:
        topk_ids = _empty((T, topk), torch.int32, logits.device, stream)
    else:
        _need(topk_ids, "topk_ids", torch.int32, 2)
        if tuple(topk_ids.shape) != (T, topk):
            raise ValueError("topk_ids must be [T, topk]")
    if topk_weights is None:
        topk_weights = _empty((T, topk), torch.float32, logits.device, stream)
    else:
        _need(topk_weights, "topk_weights", torch.float32, 2)
        if tuple(topk_weights.shape) != (T, topk):
            raise ValueError("topk_weights must be [T, topk]")
    rc = lib().mxfp4_moe_router_scored(_addr(logits), _addr(bias), T, E, topk, SCORES[scoring],
                                       n_group, topk_group, group_top, int(bool(renormalise)),
                                       route_scale, _addr(topk_ids), _addr(topk_weights),
                                       _raw_stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_router_scored")
    return topk_ids, topk_weights


def _given(t: Optional[torch.Tensor], name: str, dtype, shape):
    """``_need`` and the shape, for a tensor that may be left out."""
    if t is not None:
        _need(t, name, dtype, len(shape))
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _want(t: Optional[torch.Tensor], name: str, dtype, shape, dev: int):
    """``_given``, on the current device too (the library launches there). One expression where all is
    well: a small call's time is the host's, and a gradient's call has a dozen tensors."""
    if t is None or (type(t) is torch.Tensor and t.dtype == dtype and t.shape == shape
                     and t.is_contiguous() and t.get_device() == dev):
        return
    _given(t, name, dtype, shape)
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")


def _first(t: torch.Tensor, name: str, dtype) -> int:
    """``_need`` for the matrix that sets a call's sizes; the current device's index."""
    _need(t, name, dtype, 2)
    dev = torch._C._cuda_getDevice()
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    return dev


def _like(t: torch.Tensor, stream) -> torch.Tensor:
    """``_empty`` of t's shape and type."""
    if stream is None:
        return torch.empty_like(t)
    return _empty(t.shape, t.dtype, t.device, stream)


def _scratch(nbytes: int, workspace: Optional[torch.Tensor], device, stream, dev: int) -> torch.Tensor:
    if workspace is None:
        return _empty(nbytes, torch.uint8, device, stream)
    _need(workspace, "workspace", torch.uint8, 1)
    if workspace.get_device() != dev:
        raise ValueError("workspace must be on the current CUDA device")
    return workspace


GATE_ACTS = {"linear": 0, "sigmoid": 1}


GATE_PER = {"channel": 1, "token": 2, "value": 3}


def _gate(gate: Optional[torch.Tensor], gate_act: str, T: int, K: int, dev: int, per: Optional[str] = None):
    """(kind, activation) of a gate: bf16 [1, K], fp32 [T, 1] or bf16 [T, K], as its shape or ``per`` says."""
    if gate_act not in GATE_ACTS:
        raise ValueError(f"gate_act must be one of {sorted(GATE_ACTS)}")
    if per is not None:
        if per not in GATE_PER:
            raise ValueError(f"gate_per must be None or one of {sorted(GATE_PER)}")
        if gate is None:
            raise ValueError("gate_per needs gate")
        kind = GATE_PER[per]
        if kind == 2:
            _want(gate, "gate", torch.float32, (T, 1), dev)
        else:
            _want(gate, "gate", torch.bfloat16, (T if kind == 3 else 1, K), dev)
        return kind, GATE_ACTS[gate_act]
    if gate is None:
        return 0, GATE_ACTS[gate_act]
    if not isinstance(gate, torch.Tensor):
        raise TypeError("gate must be a torch.Tensor")
    if gate.dtype == torch.float32:
        _want(gate, "gate (fp32)", torch.float32, (T, 1), dev)
        return 2, GATE_ACTS[gate_act]
    _need(gate, "gate", torch.bfloat16, 2)
    if gate.shape[1] != K or gate.shape[0] not in (1, T):
        raise ValueError("gate must be bf16 [1, K], bf16 [T, K] or fp32 [T, 1]")
    if gate.get_device() != dev:
        raise ValueError("gate must be on the current CUDA device")
    return (1 if gate.shape[0] == 1 else 3), GATE_ACTS[gate_act]


class SandwichNorm(NamedTuple):
    """What ``sandwich_norm`` returns; what was not asked for is None."""
    y: Optional[torch.Tensor]            # bf16 [T, K]
    h: torch.Tensor                      # bf16 [T, K], the new residual stream
    q: Optional[torch.Tensor]            # y in MXFP8: E4M3 [T, K] ...
    q_scale: Optional[torch.Tensor]      # ... and E8M0 bytes [T, K/32]
    rstd: Optional[torch.Tensor]         # fp32 [2, T], both norms' factors
    x8: Optional[torch.Tensor]           # x and h in MXFP8, for the backward pass
    x8_scale: Optional[torch.Tensor]
    h8: Optional[torch.Tensor]
    h8_scale: Optional[torch.Tensor]


def sandwich_norm(x: torch.Tensor, residual: torch.Tensor, post_gamma: Optional[torch.Tensor] = None,
                  pre_gamma: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                  gate_act: str = "linear", residual_scale: Optional[torch.Tensor] = None,
                  eps: float = 1e-5, out8: Optional[str] = None, bf16: bool = True,
                  checkpoint8: Optional[str] = None, rstd: bool = False,
                  residual_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  stream=None, gate_per: Optional[str] = None) -> SandwichNorm:
    """The norm after a block, its gate, the scaled residual and the next block's norm, for bf16 rows
    [T, K]: n = x * rsqrt(mean(x^2) + eps) * post_gamma, h = residual_scale * residual + g * n,
    y = h * rsqrt(mean(h^2) + eps) * pre_gamma.

    Without post_gamma n = x; without pre_gamma there is no y. gate: bf16 [1, K] (a
    channel's), fp32 [T, 1] (a token's) or bf16 [T, K]; with one row a bf16 gate is a channel's
    unless gate_per ("channel", "token" or "value") says otherwise, as a batch of any size should. g is the gate, or its sigmoid with gate_act "sigmoid". residual_scale fp32 [1]. residual_out
    may be x or residual. out8 and bf16 as in ``add_rmsnorm``. For
    ``sandwich_norm_backward``: rstd True keeps both norms' factors, checkpoint8 "ocp" or "nosat"
    writes x and the unrounded h in MXFP8 beside the rest."""
    dev = _first(x, "x", torch.bfloat16)
    shape = x.shape
    T, K = shape
    if residual is None:
        raise TypeError("residual must be a torch.Tensor")
    _want(residual, "residual", torch.bfloat16, shape, dev)
    _want(post_gamma, "post_gamma", torch.bfloat16, (K,), dev)
    _want(pre_gamma, "pre_gamma", torch.bfloat16, (K,), dev)
    _want(residual_scale, "residual_scale", torch.float32, (1,), dev)
    _want(residual_out, "residual_out", torch.bfloat16, shape, dev)
    kind, act = _gate(gate, gate_act, T, K, dev, gate_per)
    for name, rule in (("out8", out8), ("checkpoint8", checkpoint8)):
        if rule is not None and rule not in MX8_RULES:
            raise ValueError(f"{name} must be None or one of {sorted(MX8_RULES)}")
    if pre_gamma is None:
        if out8 is not None or out is not None:
            raise ValueError("out and out8 need pre_gamma")
        bf16 = False
    if out is not None:
        if not bf16:
            raise ValueError("out is not written when bf16 is False")
        _want(out, "out", torch.bfloat16, shape, dev)
    device = x.device
    if residual_out is None:
        residual_out = _like(x, stream)
    if out is None and bf16:
        out = _like(x, stream)
    q = qs = x8 = xs = h8 = hs = r = None
    if out8 is not None:
        q = _empty(shape, torch.float8_e4m3fn, device, stream)
        qs = _empty((T, K // 32), torch.uint8, device, stream)
    if checkpoint8 is not None:
        x8 = _empty(shape, torch.float8_e4m3fn, device, stream)
        xs = _empty((T, K // 32), torch.uint8, device, stream)
        h8 = _like(x8, stream)
        hs = _like(xs, stream)
    if rstd:
        r = _empty((2, T), torch.float32, device, stream)
    rc = lib().mxfp4_moe_sandwich_norm(
        _addr(x), _addr(residual), _addr(post_gamma), _addr(pre_gamma), _addr(gate), kind, act,
        _addr(residual_scale), T, K, eps, MX8_RULES[out8 or "ocp"], MX8_RULES[checkpoint8 or "ocp"],
        _addr(residual_out), _addr(out), _addr(q), _addr(qs), _addr(x8), _addr(xs), _addr(h8),
        _addr(hs), _addr(r), _raw_stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_sandwich_norm")
    return SandwichNorm(out, residual_out, q, qs, r, x8, xs, h8, hs)


class SandwichNormGrads(NamedTuple):
    """What ``sandwich_norm_backward`` returns; None where the forward call had no such input."""
    x: torch.Tensor                           # bf16 [T, K]
    residual: torch.Tensor                    # bf16 [T, K]
    post_gamma: Optional[torch.Tensor]        # fp32 [K]
    pre_gamma: Optional[torch.Tensor]         # fp32 [K]
    gate: Optional[torch.Tensor]              # fp32 [1, K], fp32 [T, 1] or bf16 [T, K]
    residual_scale: Optional[torch.Tensor]    # fp32 [1], where residual was given


def sandwich_norm_backward_workspace_size(T: int, K: int) -> int:
    """Bytes of scratch that ``sandwich_norm_backward`` needs; 0 also for sizes it does not take."""
    return int(lib().mxfp4_moe_sandwich_norm_backward_workspace_size(T, K))


def sandwich_norm_backward(grad_h: Optional[torch.Tensor], grad_y: Optional[torch.Tensor],
                           x: torch.Tensor, h: Optional[torch.Tensor], rstd: Optional[torch.Tensor],
                           post_gamma: Optional[torch.Tensor] = None,
                           pre_gamma: Optional[torch.Tensor] = None,
                           gate: Optional[torch.Tensor] = None, gate_act: str = "linear",
                           residual: Optional[torch.Tensor] = None,
                           residual_scale: Optional[torch.Tensor] = None,
                           x_scale: Optional[torch.Tensor] = None,
                           h_scale: Optional[torch.Tensor] = None,
                           grad_x: Optional[torch.Tensor] = None,
                           grad_residual: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None,
                           stream=None, gate_per: Optional[str] = None) -> SandwichNormGrads:
    """Gradient of ``sandwich_norm`` from the gradients of its h and y (bf16 [T, K], either None) and
    from what it kept: x and h in bf16, or as x8 / h8 with x_scale / h_scale, and rstd [2, T]. h is
    needed with grad_y, rstd with grad_y or post_gamma. gate, gate_act, gate_per, gammas and residual_scale as
    in the forward call; with residual (its bf16 rows) residual_scale gets a gradient too.
    grad_x and grad_residual may be given as outputs that overlap no input."""
    dev = _first(x, "x", torch.bfloat16 if x_scale is None else torch.float8_e4m3fn)
    shape = x.shape
    T, K = shape
    if grad_h is None and grad_y is None:
        raise ValueError("grad_h or grad_y is needed")
    _want(grad_h, "grad_h", torch.bfloat16, shape, dev)
    _want(grad_y, "grad_y", torch.bfloat16, shape, dev)
    _want(post_gamma, "post_gamma", torch.bfloat16, (K,), dev)
    _want(pre_gamma, "pre_gamma", torch.bfloat16, (K,), dev)
    if grad_y is not None and (pre_gamma is None or h is None):
        raise ValueError("grad_y needs pre_gamma and h")
    _want(h, "h", torch.bfloat16 if h_scale is None else torch.float8_e4m3fn, shape, dev)
    _want(x_scale, "x_scale", torch.uint8, (T, K // 32), dev)
    _want(h_scale, "h_scale", torch.uint8, (T, K // 32), dev)
    if h is None and h_scale is not None:
        raise ValueError("h_scale needs h")
    if rstd is None and (grad_y is not None or post_gamma is not None):
        raise ValueError("rstd is needed with grad_y or post_gamma")
    _want(rstd, "rstd", torch.float32, (2, T), dev)
    _want(residual_scale, "residual_scale", torch.float32, (1,), dev)
    if residual is not None and residual_scale is None:
        raise ValueError("residual is read for residual_scale's gradient")
    _want(residual, "residual", torch.bfloat16, shape, dev)
    _want(grad_x, "grad_x", torch.bfloat16, shape, dev)
    _want(grad_residual, "grad_residual", torch.bfloat16, shape, dev)
    kind, act = _gate(gate, gate_act, T, K, dev, gate_per)
    device = x.device
    rows = grad_h if grad_h is not None else grad_y
    if grad_x is None:
        grad_x = _like(rows, stream)
    if grad_residual is None:
        grad_residual = _like(rows, stream)
    dpost = dpre = dgate = dscale = None
    if post_gamma is not None:
        dpost = _empty(K, torch.float32, device, stream)
    if pre_gamma is not None:
        dpre = _empty(K, torch.float32, device, stream)
    if kind == 1:
        dgate = _empty((1, K), torch.float32, device, stream)
    elif kind:
        dgate = _like(gate, stream)
    if residual is not None:
        dscale = _empty(1, torch.float32, device, stream)
    L = lib()
    ws = _scratch(L.mxfp4_moe_sandwich_norm_backward_workspace_size(T, K), workspace, device, stream, dev)
    rc = L.mxfp4_moe_sandwich_norm_backward(
        _addr(grad_h), _addr(grad_y), x.data_ptr(), _addr(x_scale), _addr(h), _addr(h_scale),
        _addr(rstd), _addr(post_gamma), _addr(pre_gamma), _addr(gate), kind, act, _addr(residual),
        _addr(residual_scale), T, K, grad_x.data_ptr(), grad_residual.data_ptr(), _addr(dpost),
        _addr(dpre), _addr(dgate), _addr(dscale), ws.data_ptr(), ws.numel(), _raw_stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_sandwich_norm_backward")
    return SandwichNormGrads(grad_x, grad_residual, dpost, dpre, dgate, dscale)


class RouterBalance(NamedTuple):
    """What ``router_balance`` returns."""
    stats: torch.Tensor     # fp32 [4]: balance loss, z loss, tokens, sequences with tokens
    counts: torch.Tensor    # int32 [S, E], routes to each expert
    prob: torch.Tensor      # fp32 [S, E], mean normalised score
    slope: torch.Tensor     # fp32 [S, E], a sequence's loss by a token's normalised score


def router_balance_workspace_size(T: int, E: int, n_seq: int = 1) -> int:
    """Bytes of scratch that ``router_balance`` needs; 0 for sizes it does not take."""
    return int(lib().mxfp4_moe_router_balance_workspace_size(T, E, n_seq))


def _routing(logits, topk_ids, scoring, seq_offsets):
    dev = _first(logits, "logits", torch.float32)
    _first(topk_ids, "topk_ids", torch.int32)
    T, E = logits.shape
    if topk_ids.shape[0] != T:
        raise ValueError("topk_ids must be [T, topk]")
    if scoring not in SCORES:
        raise ValueError(f"scoring must be one of {sorted(SCORES)}")
    S = 1
    if seq_offsets is not None:
        _need(seq_offsets, "seq_offsets", torch.int32, 1)
        S = seq_offsets.shape[0] - 1
        if S < 1:
            raise ValueError("seq_offsets must be [S + 1]")
        if seq_offsets.get_device() != dev:
            raise ValueError("seq_offsets must be on the current CUDA device")
    return T, E, topk_ids.shape[1], S, dev


def router_balance(logits: torch.Tensor, topk_ids: torch.Tensor, scoring: str = "sigmoid",
                   seq_offsets: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> RouterBalance:
    """Expert counts and balance losses of a routing (``router_scored``'s ids on fp32 logits [T, E]).

    p is a token's scores over their sum. A sequence's loss is E * sum_e (its share of the routes
    that went to e) * (its tokens' mean p_e), 1 for an even routing; stats[0] is the mean over the
    sequences, stats[1] the mean over tokens of logsumexp(logits)^2. seq_offsets int32 [S + 1]: rows
    of sequence i are seq_offsets[i] up to seq_offsets[i + 1] (not decreasing), None: one of all rows.
    Rows without an id in [0, E) (padding) or with every logit masked (NaN, -inf) do not count. p of a
    row whose every sigmoid ``router_scored`` has as 0 (no logit above -88.7) is 0."""
    T, E, k, S, dev = _routing(logits, topk_ids, scoring, seq_offsets)
    device = logits.device
    stats = _empty(4, torch.float32, device, stream)
    counts = _empty((S, E), torch.int32, device, stream)
    prob = _empty((S, E), torch.float32, device, stream)
    slope = _like(prob, stream)
    L = lib()
    ws = _scratch(L.mxfp4_moe_router_balance_workspace_size(T, E, S), workspace, device, stream, dev)
    rc = L.mxfp4_moe_router_balance(logits.data_ptr(), topk_ids.data_ptr(), T, E, k, SCORES[scoring],
                                    _addr(seq_offsets), S, stats.data_ptr(), counts.data_ptr(),
                                    prob.data_ptr(), slope.data_ptr(), ws.data_ptr(), ws.numel(),
                                    _raw_stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_router_balance")
    return RouterBalance(stats, counts, prob, slope)


def router_backward(logits: torch.Tensor, topk_ids: torch.Tensor,
                    grad_weights: Optional[torch.Tensor] = None, scoring: str = "sigmoid",
                    renormalise: bool = True, route_scale: float = 1.0,
                    grad_losses: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None,
                    slope: Optional[torch.Tensor] = None,
                    seq_offsets: Optional[torch.Tensor] = None,
                    grad_logits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient fp32 [T, E] of the logits: of ``router_scored``'s weights for the ids it chose, by
    grad_weights fp32 [T, topk], and of ``router_balance``'s two losses, by grad_losses fp32 [2] with
    that call's stats, slope and seq_offsets. Ids outside [0, E) and masked experts take no part;
    rows without a valid id get zeros. scoring, renormalise and route_scale as in ``router_scored``.
    Renormalised weights have their gradient where the largest chosen score is not 0 in fp32, the others'
    is 0 for scores below 2^-126."""
    T, E, k, S, dev = _routing(logits, topk_ids, scoring, seq_offsets)
    if grad_weights is None and grad_losses is None:
        raise ValueError("grad_weights or grad_losses is needed")
    _want(grad_weights, "grad_weights", torch.float32, (T, k), dev)
    if grad_losses is not None:
        if stats is None or slope is None:
            raise ValueError("grad_losses need stats and slope")
        _want(grad_losses, "grad_losses", torch.float32, (2,), dev)
        _want(stats, "stats", torch.float32, (4,), dev)
        _want(slope, "slope", torch.float32, (S, E), dev)
    if grad_logits is None:
        grad_logits = _like(logits, stream)
    else:
        _want(grad_logits, "grad_logits", torch.float32, (T, E), dev)
    rc = lib().mxfp4_moe_router_backward(
        logits.data_ptr(), topk_ids.data_ptr(), _addr(grad_weights), T, E, k, SCORES[scoring],
        int(bool(renormalise)), route_scale, _addr(grad_losses), _addr(stats), _addr(slope),
        _addr(seq_offsets), S, grad_logits.data_ptr(), _raw_stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_router_backward")
    return grad_logits


def combine_backward(grad_out: torch.Tensor, routes: torch.Tensor,
                     topk_ids: Optional[torch.Tensor] = None,
                     topk_weights: Optional[torch.Tensor] = None, routes_too: bool = False,
                     expert_base: int = 0, n_experts: int = 0,
                     grad_routes: Optional[torch.Tensor] = None, stream=None):
    """Gradient of y_t = sum_j w_tj o_tj by its weights and its routes' outputs o, bf16 [T * topk, K]
    (``forward_window(per_route=True)``): (fp32 [T, topk], and with routes_too bf16 [T * topk, K],
    else None). The latter is for routes that come from something that trains: the MXFP4 experts have no gradient. topk is topk_ids' or topk_weights' second size. Routes with a negative id, or
    outside expert_base .. expert_base + n_experts - 1 when n_experts is not 0, are skipped: gradients
    0. topk_weights fp32 [T, topk] are needed with routes_too only. grad_routes may be given as an output
    that overlaps no input."""
    dev = _first(grad_out, "grad_out", torch.bfloat16)
    _first(routes, "routes", torch.bfloat16)
    T, K = grad_out.shape
    if topk_ids is None and topk_weights is None:
        raise ValueError("topk_ids or topk_weights are needed")
    k = (topk_ids if topk_ids is not None else topk_weights).shape[-1]
    _want(topk_ids, "topk_ids", torch.int32, (T, k), dev)
    _want(topk_weights, "topk_weights", torch.float32, (T, k), dev)
    _want(routes, "routes", torch.bfloat16, (T * k, K), dev)
    if grad_routes is not None:
        routes_too = True
        _want(grad_routes, "grad_routes", torch.bfloat16, (T * k, K), dev)
    if routes_too and topk_weights is None:
        raise ValueError("routes_too needs topk_weights")
    dw = _empty((T, k), torch.float32, grad_out.device, stream) if topk_weights is None \
        else _like(topk_weights, stream)
    if routes_too and grad_routes is None:
        grad_routes = _like(routes, stream)
    rc = lib().mxfp4_moe_combine_backward(
        grad_out.data_ptr(), routes.data_ptr(), _addr(topk_ids), _addr(topk_weights), T, K, k,
        int(expert_base), int(n_experts), dw.data_ptr(), _addr(grad_routes), _raw_stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_combine_backward")
    return dw, grad_routes


def linear_workspace_size(T: int, K: int, N: int, rank: int = 0, x_is_mxfp8: bool = False) -> int:
    """Bytes of scratch that ``linear`` needs (rank 0: no adapters); 0 also for sizes it does not take."""
    return int(lib().mxfp4_moe_linear_workspace_size(T, K, N, rank, int(bool(x_is_mxfp8))))


def linear(x: torch.Tensor, w: torch.Tensor, s: torch.Tensor,
           x_scale: Optional[torch.Tensor] = None, adapter_ids: Optional[torch.Tensor] = None,
           adapter_a: Optional[torch.Tensor] = None, adapter_b: Optional[torch.Tensor] = None,
           adapter_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
           workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
           stream=None) -> torch.Tensor:
    """y[T, N] bf16 = W x_t + adapter_scale[a] * B[a] (A[a] x_t), a = adapter_ids[t].

    W is packed MXFP4: w uint8 [N, K/2], s uint8 [N, K/32]. x is bf16 [T, K], or
    float8_e4m3fn [T, K] with E8M0 bytes x_scale [T, K/32] (``add_rmsnorm``'s
    out8). adapter_ids int32 [T] (negative: none for this token), adapter_a bf16
    [L, rank, K], adapter_b bf16 [L, N, rank], adapter_scale fp32 [L] or None
    (1); without adapter_ids the plain projection. status int32 [4]: [0] counts
    the ids >= L (no adapter), [2] is non-zero when a bounded wait gave up."""
    x8 = x_scale is not None
    _need(x, "x", torch.float8_e4m3fn if x8 else torch.bfloat16, 2)
    _need(w, "w", torch.uint8, 2)
    _need(s, "s", torch.uint8, 2)
    T, K = x.shape
    N, half = w.shape
    if 2 * half != K or tuple(s.shape) != (N, K // 32):
        raise ValueError("w / s shapes must be [N, K/2] / [N, K/32]")
    if x8:
        _need(x_scale, "x_scale", torch.uint8, 2)
        if tuple(x_scale.shape) != (T, K // 32):
            raise ValueError("x_scale must be [T, K/32]")
    n_ad = rank = 0
    if adapter_ids is not None:
        _need(adapter_ids, "adapter_ids", torch.int32, 1)
        if adapter_a is None or adapter_b is None:
            raise ValueError("adapter_ids need adapter_a and adapter_b")
        _need(adapter_a, "adapter_a", torch.bfloat16, 3)
        _need(adapter_b, "adapter_b", torch.bfloat16, 3)
        n_ad, rank, ka = adapter_a.shape
        if adapter_ids.shape[0] != T:
            raise ValueError("adapter_ids must be [T]")
        if ka != K or tuple(adapter_b.shape) != (n_ad, N, rank):
            raise ValueError("adapter_a / adapter_b must be [L, rank, K] / [L, N, rank]")
        if adapter_scale is not None:
            _need(adapter_scale, "adapter_scale", torch.float32, 1)
            if adapter_scale.shape[0] != n_ad:
                raise ValueError("adapter_scale must be [L]")
    elif adapter_a is not None or adapter_b is not None or adapter_scale is not None:
        raise ValueError("adapters need adapter_ids")
    if out is None:
        out = _empty((T, N), torch.bfloat16, x.device, stream)
    else:
        _need(out, "out", torch.bfloat16, 2)
        if tuple(out.shape) != (T, N):
            raise ValueError("out must be [T, N]")
    if status is not None:
        _need(status, "status", torch.int32, 1)
        if status.shape[0] < 4:
            raise ValueError("status must be [4]")
    L = lib()
    if workspace is None:
        nbytes = L.mxfp4_moe_linear_workspace_size(T, K, N, rank, x8)
        if nbytes:
            workspace = _empty(nbytes, torch.uint8, x.device, stream)
    else:
        _need(workspace, "workspace", torch.uint8, 1)
    rc = L.mxfp4_moe_linear(x.data_ptr(), _addr(x_scale), w.data_ptr(), s.data_ptr(), T, K, N,
                            _addr(adapter_ids), _addr(adapter_a), _addr(adapter_b),
                            _addr(adapter_scale), n_ad, rank, out.data_ptr(), _addr(status),
                            _addr(workspace), 0 if workspace is None else workspace.numel(),
                            _raw_stream(stream))
    if rc:
        raise MoEError(rc, "mxfp4_moe_linear")
    return out


def set_phase_events(events) -> None:
    """Profiling hook: list of torch.cuda.Event (>= 3) recorded around each
    kernel of later forward calls, or None to disable."""
    L = lib()
    if events is None:
        L.mxfp4_moe_set_phase_events(None, 0)
        set_phase_events._keep = None
        return
    for e in events:
        if e.cuda_event == 0:     # torch creates the CUDA event on first record
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    set_phase_events._keep = arr   # the library keeps the pointer
    L.mxfp4_moe_set_phase_events(ctypes.cast(arr, ctypes.c_void_p), len(events))
