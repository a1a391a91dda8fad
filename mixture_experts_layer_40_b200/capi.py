"""ctypes binding of the C ABI in include/moe_capi.h (libmoe_b200.so).

Argument marshalling only: every function takes torch tensors (device
memory), checks dtype / contiguity / device, and passes raw pointers, sizes
and the current CUDA stream to the library function of the same name. No
computation happens here, and there is no fallback: if the library is
missing, importing this module raises.
"""
from __future__ import annotations

import bisect
import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_b200.so")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", -1: "MOE_ERR_SHAPE", -2: "MOE_ERR_NULL", -3: "MOE_ERR_CUDA",
                -4: "MOE_ERR_TIMEOUT", -5: "MOE_ERR_BOUNDS", -6: "MOE_ERR_WORKSPACE",
                -7: "MOE_ERR_ALIGN"}


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {STATUS_NAMES.get(code, code)}")
        self.code = code


class moe_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32), ("I", ctypes.c_int32), ("G", ctypes.c_int32),
                ("M", ctypes.c_int32)]


class moe_weights(ctypes.Structure):
    _fields_ = [("gate_w", ctypes.c_void_p), ("w13", ctypes.c_void_p), ("s13", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("s2", ctypes.c_void_p), ("gate_split", ctypes.c_void_p)]


class moe_grad_list(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("grads", ctypes.POINTER(ctypes.c_void_p)),
                ("out", ctypes.POINTER(ctypes.c_void_p)), ("sizes", ctypes.POINTER(ctypes.c_int64)),
                ("types", ctypes.POINTER(ctypes.c_int32)), ("table", ctypes.c_void_p),
                ("plan", ctypes.c_int32 * 4)]


_LAYOUT_FIELDS = ["status", "counts", "offsets", "group_rows", "row_start", "row_token",
                  "token_row", "topk_ids", "topk_gates", "logits", "a_q", "a_s", "h_q", "h_s",
                  "y_rows", "gate_split", "bal_scratch", "perm_scratch", "total"]


class moe_ws_layout(ctypes.Structure):
    _fields_ = ([("routed_cap", ctypes.c_int64), ("rows_total", ctypes.c_int64)]
                + [(f, ctypes.c_size_t) for f in _LAYOUT_FIELDS])


# name -> (restype, argtypes) of every function declared in the header
_P = ctypes.c_void_p
_I32, _I64, _F32, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "moe_quantize_1x128": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P]),
    "moe_quantize_128x128": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P]),
    "moe_workspace_size": (_SZ, [moe_shape]),
    "moe_workspace_layout": (ctypes.c_int, [moe_shape, ctypes.POINTER(moe_ws_layout)]),
    "moe_split_gate": (ctypes.c_int, [_P, _I32, _I32, _P, _P]),
    "moe_route": (ctypes.c_int, [moe_shape, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_route_noalloc": (ctypes.c_int, [moe_shape, _P, _P, _P, _P, _P, _P, _P]),
    "moe_balance_stats": (ctypes.c_int, [moe_shape, ctypes.c_int32, ctypes.c_float, _P, _SZ, _P,
                                         _P, _P, _P, _P]),
    "moe_transpose_weights": (ctypes.c_int, [moe_shape, ctypes.POINTER(moe_weights), _P, _P, _P,
                                             _P, _P]),
    "moe_backward_workspace_size": (_SZ, [moe_shape]),
    "moe_backward": (ctypes.c_int, [moe_shape, ctypes.POINTER(moe_weights),
                                    ctypes.POINTER(moe_weights), _P, _P, _P, _P, _P, _SZ, _P, _SZ,
                                    _P, _P, _P, _P, _P]),
    "moe_forward": (ctypes.c_int, [moe_shape, ctypes.POINTER(moe_weights), _P, _P, _P, _P, _P, _P,
                                   _P, _SZ, _P]),
    "moe_forward_traced": (ctypes.c_int, [moe_shape, ctypes.POINTER(moe_weights), _P, _P, _P, _P,
                                          _P, _P, _P, _SZ, _P, ctypes.POINTER(_P), _I32]),
    "moe_update_bias": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, _F32, _P]),
    "moe_expert_up": (ctypes.c_int, [_I32, _I32, _I32, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_expert_down": (ctypes.c_int, [_I32, _I32, _I32, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _P]),
    "moe_expert_down_bf16": (ctypes.c_int, [_I32, _I32, _I32, _P, _P, _I64, _P, _P, _P, _P, _P, _P,
                                            _P]),
    "moe_grouped_matmul": (ctypes.c_int, [_I32, _I32, _I32, _P, _P, _I64, _I32, _I32, _P, _P, _I32,
                                          _P, _P, _P]),
    "moe_grouped_wgrad": (ctypes.c_int, [_I32, _I32, _I32, _P, _P, _I64, _I32, _I32, _P, _P, _P,
                                         _I32, _P, _P]),
    "moe_block_norm": (ctypes.c_int, [_I64, _I32, _I32, _I32, _I32, _I32, _F32, _F32, _P, _P, _P,
                                      _P, _P, _P, _P, _P, _P]),
    "moe_block_norm_backward_workspace_size": (_SZ, [_I32]),
    "moe_block_norm_backward": (ctypes.c_int, [_I64, _I32, _I32, _I32, _I32, _I32, _F32, _F32, _P,
                                               _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                               _P, _SZ, _P]),
    "moe_grad_table_size": (_SZ, [ctypes.POINTER(moe_grad_list)]),
    "moe_grad_table": (ctypes.c_int, [ctypes.POINTER(moe_grad_list), _P]),
    "moe_grad_sumsq": (ctypes.c_int, [ctypes.POINTER(moe_grad_list), _P, _P]),
    "moe_grad_clip": (ctypes.c_int, [ctypes.POINTER(moe_grad_list), _P, _F32, _P, _P]),
    "moe_ep_row_bytes": (_I64, [moe_shape]),
    "moe_ep_dispatch_workspace_size": (_SZ, [moe_shape, _I32]),
    "moe_ep_dispatch": (ctypes.c_int, [moe_shape, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _P,
                                       _P, _SZ, _P]),
    "moe_ep_shared": (ctypes.c_int, [moe_shape, _I32, ctypes.POINTER(moe_weights), _P, _SZ, _P]),
    "moe_ep_expert_workspace_size": (_SZ, [moe_shape, _I32, _I64, _I64]),
    "moe_ep_experts": (ctypes.c_int, [moe_shape, _I32, ctypes.POINTER(moe_weights), _P, _I64,
                                      _I64, _P, _P, _SZ, _P]),
    "moe_ep_combine": (ctypes.c_int, [moe_shape, _I32, _P, _I64, _P, _SZ, _P, _P]),
    "moe_ep_peer_expert_workspace_size": (_SZ, [moe_shape, _I32, _I32]),
    "moe_ep_dispatch_peer": (ctypes.c_int, [moe_shape, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P,
                                            _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_ep_experts_peer": (ctypes.c_int, [moe_shape, _I32, _I32, _I32,
                                           ctypes.POINTER(moe_weights), _P, _P, _P, _P, _SZ, _P]),
    "moe_ep_combine_peer": (ctypes.c_int, [moe_shape, _I32, _I32, _P, _P, _SZ, _P, _P]),
    "moe_get_status": (ctypes.c_int, [_P, _P]),
    "moe_device_sm_count": (ctypes.c_int, []),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m mixture_experts_layer_40_b200.build` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


LIB = _load()


def _check(name: str, code: int) -> None:
    if code != MOE_OK:
        raise MoeError(name, code)


def _ptr(t: torch.Tensor | None, dtype: torch.dtype | None = None, name: str = "tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def shape_of(T: int, H: int, N: int, K: int, I: int, G: int = 0, M: int = 0) -> moe_shape:
    """G, M: node-limited routing over G expert groups, M per token (G = 0: off)."""
    return moe_shape(T, H, N, K, I, G, M)


def moe_quantize_1x128(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, stream=None):
    rows, cols = x.shape
    _check("moe_quantize_1x128", LIB.moe_quantize_1x128(
        _ptr(x, torch.bfloat16, "x"), rows, cols, _ptr(q, torch.uint8, "q"),
        _ptr(scales, torch.float32, "scales"), _stream(stream)))


def moe_quantize_128x128(w: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, stream=None):
    rows, cols = w.shape
    _check("moe_quantize_128x128", LIB.moe_quantize_128x128(
        _ptr(w, torch.float32, "w"), rows, cols, _ptr(q, torch.uint8, "q"),
        _ptr(scales, torch.float32, "scales"), _stream(stream)))


def moe_workspace_size(sh: moe_shape) -> int:
    return int(LIB.moe_workspace_size(sh))


def moe_workspace_layout(sh: moe_shape) -> moe_ws_layout:
    out = moe_ws_layout()
    _check("moe_workspace_layout", LIB.moe_workspace_layout(sh, ctypes.byref(out)))
    return out


def moe_route(sh: moe_shape, gate_w, x, bias, topk_ids, topk_gates, counts, ws, stream=None):
    _check("moe_route", LIB.moe_route(
        sh, _ptr(gate_w, torch.float32, "gate_w"), _ptr(x, torch.bfloat16, "x"),
        _ptr(bias, torch.float32, "bias"), _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(topk_gates, torch.float32, "topk_gates"), _ptr(counts, torch.int32, "counts"),
        _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))


def moe_balance_stats(sh: moe_shape, seq_len: int, alpha: float, ws, topk_ids, f, P, loss,
                      stream=None):
    """Sequence-wise balance statistics of the routing the last moe_route /
    moe_forward on `ws` made: f, P float [S, N], loss float [S]."""
    _check("moe_balance_stats", LIB.moe_balance_stats(
        sh, seq_len, alpha, _ptr(ws, torch.uint8, "ws"), ws.numel(),
        _ptr(topk_ids, torch.int32, "topk_ids"), _ptr(f, torch.float32, "f"),
        _ptr(P, torch.float32, "P"), _ptr(loss, torch.float32, "loss"), _stream(stream)))


def moe_transpose_weights(sh: moe_shape, w: moe_weights, w13t, s13t, w2t, s2t, stream=None):
    _check("moe_transpose_weights", LIB.moe_transpose_weights(
        sh, ctypes.byref(w), _ptr(w13t, torch.uint8, "w13t"), _ptr(s13t, torch.float32, "s13t"),
        _ptr(w2t, torch.uint8, "w2t"), _ptr(s2t, torch.float32, "s2t"), _stream(stream)))


def moe_backward_workspace_size(sh: moe_shape) -> int:
    return int(LIB.moe_backward_workspace_size(sh))


def moe_backward(sh: moe_shape, w: moe_weights, wt: moe_weights, topk_ids, topk_gates, x, dy, ws,
                 bws, dx, dgates, dw13=None, dw2=None, stream=None):
    _check("moe_backward", LIB.moe_backward(
        sh, ctypes.byref(w), ctypes.byref(wt), _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(topk_gates, torch.float32, "topk_gates"), _ptr(x, torch.bfloat16, "x"),
        _ptr(dy, torch.bfloat16, "dy"), _ptr(ws, torch.uint8, "ws"), ws.numel(),
        _ptr(bws, torch.uint8, "bws"), bws.numel(), _ptr(dx, torch.bfloat16, "dx"),
        _ptr(dgates, torch.float32, "dgates"), _ptr(dw13, torch.float32, "dw13"),
        _ptr(dw2, torch.float32, "dw2"), _stream(stream)))


ROUTE_NOALLOC_MAX_LOGITS = 1048576


def moe_route_noalloc(sh: moe_shape, gate_w, x, bias, topk_ids, topk_gates, counts, stream=None):
    """moe_route without a workspace: the logits scratch is a fixed 4 MiB array
    inside the library (T * N <= ROUTE_NOALLOC_MAX_LOGITS). For callers that
    cannot give the library device memory; calls must not overlap on the GPU."""
    _check("moe_route_noalloc", LIB.moe_route_noalloc(
        sh, _ptr(gate_w, torch.float32, "gate_w"), _ptr(x, torch.bfloat16, "x"),
        _ptr(bias, torch.float32, "bias"), _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(topk_gates, torch.float32, "topk_gates"), _ptr(counts, torch.int32, "counts"),
        _stream(stream)))


def make_weights(gate_w, w13, s13, w2, s2, gate_split=None) -> moe_weights:
    return moe_weights(_ptr(gate_w, torch.float32, "gate_w"), _ptr(w13, torch.uint8, "w13"),
                       _ptr(s13, torch.float32, "s13"), _ptr(w2, torch.uint8, "w2"),
                       _ptr(s2, torch.float32, "s2"),
                       None if gate_split is None else _ptr(gate_split, torch.bfloat16,
                                                            "gate_split"))


def _check_split_size(gate_split, N: int, H: int) -> None:
    # the three bf16 terms are written (moe_split_gate) or read whole
    if gate_split is not None and gate_split.numel() < 3 * N * H:
        raise ValueError(f"gate_split holds {gate_split.numel()} values; the three terms of "
                         f"[{N}, {H}] centroids need {3 * N * H}")


def moe_split_gate(gate_w, gate_split, stream=None):
    N, H = gate_w.shape
    _check_split_size(gate_split, N, H)
    _check("moe_split_gate", LIB.moe_split_gate(
        _ptr(gate_w, torch.float32, "gate_w"), N, H, _ptr(gate_split, torch.bfloat16, "gate_split"),
        _stream(stream)))


def moe_forward(sh: moe_shape, w: moe_weights, x, bias, y, topk_ids=None, topk_gates=None,
                counts=None, ws=None, stream=None):
    _check("moe_forward", LIB.moe_forward(
        sh, ctypes.byref(w), _ptr(x, torch.bfloat16, "x"), _ptr(bias, torch.float32, "bias"),
        _ptr(y, torch.bfloat16, "y"), _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(topk_gates, torch.float32, "topk_gates"), _ptr(counts, torch.int32, "counts"),
        _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))


TRACE_EVENTS = 7
TRACE_STAGES = ["route", "permute", "quantize", "expert_up", "expert_down", "combine"]


def moe_forward_traced(sh: moe_shape, w: moe_weights, x, bias, y, events, topk_ids=None,
                       topk_gates=None, counts=None, ws=None, stream=None):
    """moe_forward that also records `events` (TRACE_EVENTS torch.cuda.Event
    objects created with enable_timing=True) around its six stages."""
    arr = (_P * len(events))(*[ev.cuda_event for ev in events])
    _check("moe_forward_traced", LIB.moe_forward_traced(
        sh, ctypes.byref(w), _ptr(x, torch.bfloat16, "x"), _ptr(bias, torch.float32, "bias"),
        _ptr(y, torch.bfloat16, "y"), _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(topk_gates, torch.float32, "topk_gates"), _ptr(counts, torch.int32, "counts"),
        _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream), arr, len(events)))


def moe_update_bias(bias, counts, N: int, T: int, K: int, gamma: float, stream=None):
    _check("moe_update_bias", LIB.moe_update_bias(
        _ptr(bias, torch.float32, "bias"), _ptr(counts, torch.int32, "counts"), N, T, K,
        float(gamma), _stream(stream)))


def moe_expert_up(H, I, n_groups, group_rows, group_start, rows, a_q, a_s, w13, s13, h_q, h_s,
                  status, stream=None):
    _check("moe_expert_up", LIB.moe_expert_up(
        H, I, n_groups, _ptr(group_rows, torch.int32), _ptr(group_start, torch.int32), rows,
        _ptr(a_q, torch.uint8), _ptr(a_s, torch.float32), _ptr(w13, torch.uint8),
        _ptr(s13, torch.float32), _ptr(h_q, torch.uint8), _ptr(h_s, torch.float32),
        _ptr(status), _stream(stream)))


def moe_expert_down(H, I, n_groups, group_rows, group_start, rows, h_q, h_s, w2, s2, y_rows,
                    status, stream=None):
    _check("moe_expert_down", LIB.moe_expert_down(
        H, I, n_groups, _ptr(group_rows, torch.int32), _ptr(group_start, torch.int32), rows,
        _ptr(h_q, torch.uint8), _ptr(h_s, torch.float32), _ptr(w2, torch.uint8),
        _ptr(s2, torch.float32), _ptr(y_rows, torch.float32), _ptr(status), _stream(stream)))


def moe_expert_down_bf16(H, I, n_groups, group_rows, group_start, rows, h_q, h_s, w2, s2, y_rows,
                         status, stream=None):
    _check("moe_expert_down_bf16", LIB.moe_expert_down_bf16(
        H, I, n_groups, _ptr(group_rows, torch.int32), _ptr(group_start, torch.int32), rows,
        _ptr(h_q, torch.uint8), _ptr(h_s, torch.float32), _ptr(w2, torch.uint8),
        _ptr(s2, torch.float32), _ptr(y_rows, torch.bfloat16), _ptr(status), _stream(stream)))


# ------------------------------------------------- operators beside the layer
#
# These check sizes as well, since they are given no shape struct, and run on
# the device that holds their tensors: its current stream, or `stream` of it.
TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _type(t: torch.Tensor, name: str) -> int:
    if t.dtype not in TYPES:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return TYPES[t.dtype]


def _need(t: torch.Tensor | None, dtype: torch.dtype, shape: tuple, device: int, name: str):
    """The address of a tensor (or None) that must be contiguous, of this type
    and shape, on the CUDA device of this index."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    _ptr(t, dtype, name)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")


def _device(t: torch.Tensor, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _run(name: str, device: int, stream, *args) -> None:
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device)
    elif stream.device.index != device:
        raise ValueError(f"{name}: the stream is on {stream.device}, the tensors on cuda:{device}")
    else:
        handle = stream.cuda_stream
    fn = getattr(LIB, name)
    if device == torch._C._cuda_getDevice():
        code = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            code = fn(*args, handle)
    if code != MOE_OK:
        raise MoeError(name, code)


def keep_until_done(device: int, stream, *tensors) -> None:
    """The tensors' memory is not given to others before `stream` (None: the
    device's current one) is done with what it holds now, even if they are
    dropped; for tensors that a holder made on one stream and uses on another."""
    at = torch.cuda.current_stream(device) if stream is None else stream
    for t in tensors:
        if t is not None:
            t.record_stream(at)


def _sums_type(t: torch.Tensor, of: torch.Tensor, name: str) -> int:
    if t.dtype not in (of.dtype, torch.float32):
        raise ValueError(f"{name} must be {of.dtype} or float32, got {t.dtype}")
    return _type(t, name)


def _groups(group_rows, group_start, n_groups: int, device, status):
    if status is not None:
        if status.get_device() != device:
            raise ValueError(f"status must be on cuda:{device}, got {status.device}")
        if status.numel() * status.element_size() < 4:
            raise ValueError("status must hold the 4 bytes of a status word")
    return (_need(group_rows, torch.int32, (n_groups,), device, "group_rows"),
            _need(group_start, torch.int32, (n_groups,), device, "group_start"),
            _ptr(status, None, "status"))


def moe_grouped_matmul(a, b, group_rows, group_start, out, trans_b: bool = True, status=None,
                       stream=None):
    """out[r] = a[r] @ b[g]^T (trans_b; b [G, N, K]) or a[r] @ b[g] (b [G, K, N])
    for the rows r of each group g: group_rows[g] rows from group_start[g], any
    alignment. a [R, K] and b bf16 or fp16 alike; out [R, N] of their type or
    float32. Rows of out outside every group are left as they are."""
    if a.dim() != 2 or b.dim() != 3:
        raise ValueError("a must be [rows, K] and b three-dimensional")
    rows, K = a.shape
    G, N = b.shape[0], b.shape[1 if trans_b else 2]
    t = _type(a, "a")
    dev = _device(a, "a")
    ap = _need(a, a.dtype, (rows, K), dev, "a")
    bp = _need(b, a.dtype, (G, N, K) if trans_b else (G, K, N), dev, "b")
    op = _need(out, out.dtype, (rows, N), dev, "out")
    gr, gs, st = _groups(group_rows, group_start, G, dev, status)
    _run("moe_grouped_matmul", dev, stream, t, _sums_type(out, a, "out"), G, gr, gs, rows, K, N, ap, bp,
         1 if trans_b else 0, op, st)


def moe_grouped_wgrad(dy, x, group_rows, group_start, dw, accumulate: bool = False, status=None,
                      stream=None):
    """dw[g] = dy_g^T @ x_g over the rows of each group g (added to dw with
    accumulate). dy [R, N] and x [R, K] bf16 or fp16 alike; dw [G, N, K] of
    their type or float32."""
    if dy.dim() != 2 or x.dim() != 2 or dw.dim() != 3:
        raise ValueError("dy and x must be [rows, N] and [rows, K], dw three-dimensional")
    rows, N = dy.shape
    K, G = x.shape[1], dw.shape[0]
    t = _type(dy, "dy")
    dev = _device(dy, "dy")
    yp = _need(dy, dy.dtype, (rows, N), dev, "dy")
    xp = _need(x, dy.dtype, (rows, K), dev, "x")
    wp = _need(dw, dw.dtype, (G, N, K), dev, "dw")
    gr, gs, st = _groups(group_rows, group_start, G, dev, status)
    _run("moe_grouped_wgrad", dev, stream, t, _sums_type(dw, dy, "dw"), G, gr, gs, rows, N, K, yp, xp, wp,
         1 if accumulate else 0, st)


def _norm_types(x, act, pre, post, scale):
    """Type codes of the residual stream, the block and the weights, which must
    agree among themselves."""
    w = pre if pre is not None else post if post is not None else scale
    wt = act.dtype if w is None else w.dtype
    try:
        return wt, TYPES[x.dtype], TYPES[act.dtype], TYPES[wt]
    except KeyError:
        raise ValueError(f"bfloat16, float16 or float32 tensors are needed, got {x.dtype}, "
                         f"{act.dtype} and weights of {wt}") from None


def moe_block_norm(x, eps: float, pre_weight=None, u=None, z=None, post_weight=None, gate=None,
                   scale=None, alpha: float = 1.0, r=None, stream=None):
    """r = x + alpha * scale * gate * N(z; post_weight) and u = N(r; pre_weight),
    N(v; w) = v * rsqrt(mean(v^2) + eps) * w by row. Without z only u (of x);
    without pre_weight only r. x, r [T, H] bf16, fp16 or float32; z, u of the
    same type or, with x float32, any; gate float32 [T] or [T, H] of z's type;
    weights and scale [H] of z's type or float32. r may be x and u may be z."""
    if (z is None) != (r is None) or (pre_weight is None) != (u is None):
        raise ValueError("r goes with z, and u with pre_weight")
    act = u if z is None else z
    if act is None:
        raise ValueError("nothing to compute: give z and r, pre_weight and u, or both")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("the rows must be two-dimensional")
    dev = _device(x, "x")
    wt, rc, ac, wc = _norm_types(x, act, pre_weight, post_weight, scale)
    T, H = shape
    kind = 0 if gate is None else 1 if gate.dim() == 1 else 2
    res, at, cols = x.dtype, act.dtype, (H,)
    _run("moe_block_norm", dev, stream, T, H, rc, ac, wc, kind, alpha, eps,
         _need(x, res, shape, dev, "x"),
         None if z is None else _need(z, at, shape, dev, "z"),
         None if gate is None else _need(gate, torch.float32, (T,), dev, "gate") if kind == 1
         else _need(gate, at, shape, dev, "gate"),
         None if pre_weight is None else _need(pre_weight, wt, cols, dev, "pre_weight"),
         None if post_weight is None else _need(post_weight, wt, cols, dev, "post_weight"),
         None if scale is None else _need(scale, wt, cols, dev, "scale"),
         None if r is None else _need(r, res, shape, dev, "r"),
         None if u is None else _need(u, at, shape, dev, "u"))


def moe_block_norm_backward_workspace_size(H: int) -> int:
    return int(LIB.moe_block_norm_backward_workspace_size(H))


def moe_block_norm_backward(r, eps: float, ws, dr=None, du=None, pre_weight=None, z=None,
                            post_weight=None, gate=None, scale=None, alpha: float = 1.0, dx=None,
                            dz=None, dgate=None, dscale=None, dpost=None, dpre=None, stream=None):
    """Gradients of moe_block_norm for the upstream dr (of r; None: zero) and du
    (of u). r: the forward's r, or its x where it had no z. dx like r (with
    pre_weight; without it the gradient of x is dr itself), dz like z, dgate
    like gate, dpre, dpost and dscale float32 [H]. ws: uint8, at least
    moe_block_norm_backward_workspace_size(H) bytes."""
    if (z is None) != (dz is None) or (gate is None) != (dgate is None):
        raise ValueError("dz goes with z, and dgate with gate")
    if (scale is None) != (dscale is None) or (post_weight is None) != (dpost is None):
        raise ValueError("dscale goes with scale, and dpost with post_weight")
    given = pre_weight is not None
    if (dpre is not None) != given or (dx is not None) != given or (du is not None) != given:
        raise ValueError("du, dx and dpre go with pre_weight")
    act = du if z is None else z
    if act is None:
        raise ValueError("nothing to compute: give z, du or both")
    shape = r.shape
    if len(shape) != 2:
        raise ValueError("the rows must be two-dimensional")
    dev = _device(r, "r")
    wt, rc, ac, wc = _norm_types(r, act, pre_weight, post_weight, scale)
    T, H = shape
    kind = 0 if gate is None else 1 if gate.dim() == 1 else 2
    res, at, cols, f32 = r.dtype, act.dtype, (H,), torch.float32
    gt, gs = (f32, (T,)) if kind == 1 else (at, shape)
    if ws.get_device() != dev:
        raise ValueError(f"ws must be on cuda:{dev}, got {ws.device}")
    _run("moe_block_norm_backward", dev, stream, T, H, rc, ac, wc, kind, alpha, eps,
         _need(r, res, shape, dev, "r"),
         None if z is None else _need(z, at, shape, dev, "z"),
         None if gate is None else _need(gate, gt, gs, dev, "gate"),
         _need(pre_weight, wt, cols, dev, "pre_weight") if given else None,
         None if post_weight is None else _need(post_weight, wt, cols, dev, "post_weight"),
         None if scale is None else _need(scale, wt, cols, dev, "scale"),
         None if dr is None else _need(dr, res, shape, dev, "dr"),
         _need(du, at, shape, dev, "du") if given else None,
         _need(dx, res, shape, dev, "dx") if given else None,
         None if dz is None else _need(dz, at, shape, dev, "dz"),
         None if dgate is None else _need(dgate, gt, gs, dev, "dgate"),
         _need(dpre, f32, cols, dev, "dpre") if given else None,
         None if dpost is None else _need(dpost, f32, cols, dev, "dpost"),
         None if dscale is None else _need(dscale, f32, cols, dev, "dscale"),
         _ptr(ws, torch.uint8, "ws"), ws.numel())


GRAD_PARTIALS = 1024


class GradList:
    """A moe_grad_list over a program's gradient tensors, made once by
    make_grad_list (outside a graph capture) and used in every step that writes
    new gradients into them; it keeps the tensors."""

    def __init__(self, grads, out):
        self.grads, self.out = list(grads), None if out is None else list(out)
        n = len(self.grads)
        if self.out is not None and len(self.out) != n:
            raise ValueError(f"{n} gradients and {len(self.out)} outputs")
        self.device = _device(self.grads[0], "grads[0]") if n else None
        gp = [_need(g, g.dtype, g.shape, self.device, f"grads[{i}]")
              for i, g in enumerate(self.grads)]
        op = None
        if self.out is not None:
            op = [_need(o, g.dtype, g.shape, self.device, f"out[{i}]")
                  for i, (o, g) in enumerate(zip(self.out, self.grads))]
        sizes = [g.numel() for g in self.grads]
        self._refuse_overlap(gp, op, [g.numel() * g.element_size() for g in self.grads])
        ptrs = ctypes.c_void_p * n
        self._arrays = (ptrs(*gp), None if op is None else ptrs(*op),
                        (ctypes.c_int64 * n)(*sizes),
                        (ctypes.c_int32 * n)(*[_type(g, f"grads[{i}]")
                                               for i, g in enumerate(self.grads)]))
        g, o, s, t = self._arrays
        cast = ctypes.cast
        vpp = ctypes.POINTER(ctypes.c_void_p)
        self.struct = moe_grad_list(n, cast(g, vpp), None if o is None else cast(o, vpp),
                                    cast(s, ctypes.POINTER(ctypes.c_int64)),
                                    cast(t, ctypes.POINTER(ctypes.c_int32)), None)
        # longer lists read their table from device memory
        self._table = None
        nbytes = int(LIB.moe_grad_table_size(ctypes.byref(self.struct)))
        if nbytes:
            host = torch.empty(nbytes, dtype=torch.uint8)
            _check("moe_grad_table", LIB.moe_grad_table(ctypes.byref(self.struct), host.data_ptr()))
            self._table = host.to(torch.device("cuda", self.device))
            torch.cuda.current_stream(self.device).synchronize()  # for every later stream
            self.struct.table = self._table.data_ptr()

    @staticmethod
    def _refuse_overlap(grads, out, nbytes):
        """Raises ValueError where an output lies on another output or, unless
        it is the tensor itself, on gradients (addresses and sizes)."""
        written = grads if out is None else out
        spans = sorted((p, p + b, i) for i, (p, b) in enumerate(zip(written, nbytes)) if b)
        for (_, end, i), (begin, _, j) in zip(spans, spans[1:]):
            if begin < end:
                raise ValueError(f"tensors {i} and {j} overlap where they are written")
        if out is None:
            return
        ends = [end for _, end, _ in spans]
        for j, (p, b) in enumerate(zip(grads, nbytes)):
            for begin, end, i in spans[bisect.bisect_right(ends, p):]:
                if not b or begin >= p + b:
                    break
                if i != j or begin != p:
                    raise ValueError(f"the output of tensor {i} overlaps gradient {j}")


def make_grad_list(grads, out=None) -> GradList:
    """grads: contiguous bf16, fp16 or float32 tensors on one device (types may
    differ); out: tensors of the same shapes and types for the clipped
    gradients, or None to scale in place. Outputs must not overlap one another
    or another tensor's gradients (ValueError)."""
    return GradList(grads, out)


def _partials(gl: GradList, partials):
    dev = gl.device if gl.device is not None else _device(partials, "partials")
    return dev, _need(partials, torch.float64, (GRAD_PARTIALS,), dev, "partials")


def moe_grad_sumsq(gl: GradList, partials, stream=None):
    """Partial sums of squares of all gradients of the list: partials float64
    [GRAD_PARTIALS]; their sum is the squared global norm. With sharded
    experts, add the ranks' partials (an all-reduce) before moe_grad_clip."""
    dev, p = _partials(gl, partials)
    _run("moe_grad_sumsq", dev, stream, ctypes.byref(gl.struct), p)
    if gl._table is not None:
        keep_until_done(dev, stream, gl._table)


def moe_grad_clip(gl: GradList, partials, max_norm: float, norm, stream=None):
    """norm (float32 [1]) = sqrt(sum of partials); every gradient times
    min(1, max_norm / (norm + 1e-6)) into the list's outputs (or in place)."""
    dev, p = _partials(gl, partials)
    _run("moe_grad_clip", dev, stream, ctypes.byref(gl.struct), p, float(max_norm),
         _need(norm, torch.float32, (1,), dev, "norm"))
    if gl._table is not None:
        keep_until_done(dev, stream, gl._table)


def moe_ep_row_bytes(sh: moe_shape) -> int:
    return int(LIB.moe_ep_row_bytes(sh))


def moe_ep_dispatch_workspace_size(sh: moe_shape, W: int) -> int:
    return int(LIB.moe_ep_dispatch_workspace_size(sh, W))


def moe_ep_expert_workspace_size(sh: moe_shape, W: int, R: int, pairs: int) -> int:
    return int(LIB.moe_ep_expert_workspace_size(sh, W, R, pairs))


def moe_ep_dispatch(sh: moe_shape, W: int, gate_w, x, bias, send, send_counts, ws,
                    topk_ids=None, topk_gates=None, counts=None, stream=None, gate_split=None):
    """send: uint8 [send_cap, moe_ep_row_bytes(sh)]; send_counts: int32 [W, 2];
    gate_split: None, or bf16 [3, N, H] from moe_split_gate."""
    _check_split_size(gate_split, sh.N, sh.H)
    _check("moe_ep_dispatch", LIB.moe_ep_dispatch(
        sh, W, _ptr(gate_w, torch.float32, "gate_w"),
        _ptr(gate_split, torch.bfloat16, "gate_split"), _ptr(x, torch.bfloat16, "x"),
        _ptr(bias, torch.float32, "bias"), _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(topk_gates, torch.float32, "topk_gates"), _ptr(counts, torch.int32, "counts"),
        _ptr(send, torch.uint8, "send"), send.shape[0] if send is not None else 0,
        _ptr(send_counts, torch.int32, "send_counts"), _ptr(ws, torch.uint8, "ws"), ws.numel(),
        _stream(stream)))


def moe_ep_shared(sh: moe_shape, W: int, w_local: moe_weights, ws, stream=None):
    _check("moe_ep_shared", LIB.moe_ep_shared(
        sh, W, ctypes.byref(w_local), _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))


def moe_ep_experts(sh: moe_shape, W: int, w_local: moe_weights, recv, R: int, pairs: int, out, ws,
                   stream=None):
    """recv: uint8 [>= R, row_bytes]; out: float32 [>= R, H]."""
    _check("moe_ep_experts", LIB.moe_ep_experts(
        sh, W, ctypes.byref(w_local), _ptr(recv, torch.uint8, "recv"), R, pairs,
        _ptr(out, torch.float32, "out"), _ptr(ws, torch.uint8, "ws"), ws.numel(),
        _stream(stream)))


def moe_ep_combine(sh: moe_shape, W: int, ret, ret_rows: int, ws, y, stream=None):
    _check("moe_ep_combine", LIB.moe_ep_combine(
        sh, W, _ptr(ret, torch.float32, "ret"), ret_rows, _ptr(ws, torch.uint8, "ws"), ws.numel(),
        _ptr(y, torch.bfloat16, "y"), _stream(stream)))


def moe_ep_peer_expert_workspace_size(sh: moe_shape, W: int, T_cap: int) -> int:
    return int(LIB.moe_ep_peer_expert_workspace_size(sh, W, T_cap))


def moe_ep_dispatch_peer(sh: moe_shape, W: int, rank: int, T_cap: int, gate_w, x, bias,
                         peer_recv, peer_counts, ws, topk_ids=None, topk_gates=None, counts=None,
                         send_counts=None, stream=None, gate_split=None):
    """peer_recv, peer_counts: int64 device tensors [W] of device pointers;
    gate_split as in moe_ep_dispatch."""
    _check_split_size(gate_split, sh.N, sh.H)
    _check("moe_ep_dispatch_peer", LIB.moe_ep_dispatch_peer(
        sh, W, rank, T_cap, _ptr(gate_w, torch.float32, "gate_w"),
        _ptr(gate_split, torch.bfloat16, "gate_split"), _ptr(x, torch.bfloat16, "x"),
        _ptr(bias, torch.float32, "bias"), _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(topk_gates, torch.float32, "topk_gates"), _ptr(counts, torch.int32, "counts"),
        _ptr(peer_recv, torch.int64, "peer_recv"), _ptr(peer_counts, torch.int64, "peer_counts"),
        _ptr(send_counts, torch.int32, "send_counts"), _ptr(ws, torch.uint8, "ws"), ws.numel(),
        _stream(stream)))


def moe_ep_experts_peer(sh: moe_shape, W: int, rank: int, T_cap: int, w_local: moe_weights, recv,
                        recv_counts, peer_ret, ws, stream=None):
    """peer_ret: int64 device tensor [W] of device pointers."""
    _check("moe_ep_experts_peer", LIB.moe_ep_experts_peer(
        sh, W, rank, T_cap, ctypes.byref(w_local), _ptr(recv, torch.uint8, "recv"),
        _ptr(recv_counts, torch.int32, "recv_counts"), _ptr(peer_ret, torch.int64, "peer_ret"),
        _ptr(ws, torch.uint8, "ws"), ws.numel(), _stream(stream)))


def moe_ep_combine_peer(sh: moe_shape, W: int, T_cap: int, ret, ws, y, stream=None):
    _check("moe_ep_combine_peer", LIB.moe_ep_combine_peer(
        sh, W, T_cap, _ptr(ret, torch.float32, "ret"), _ptr(ws, torch.uint8, "ws"), ws.numel(),
        _ptr(y, torch.bfloat16, "y"), _stream(stream)))


def moe_get_status(ws, stream=None) -> int:
    return int(LIB.moe_get_status(_ptr(ws), _stream(stream)))


def moe_device_sm_count() -> int:
    return int(LIB.moe_device_sm_count())
