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
from typing import Optional

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
