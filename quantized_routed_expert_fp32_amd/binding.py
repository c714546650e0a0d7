"""Python binding of libmoe.so (include/moe.h): argument marshalling only.

Every step of the routed-expert FFN runs in the library's HIP kernels; this
module passes device pointers (torch tensors) and the current HIP stream.
It raises if the library is missing: there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# MOE_LIBRARY names another build of the same library (the host-only
# sanitizer flavour of the host tests); it must exist like the default one
LIB_PATH = os.environ.get("MOE_LIBRARY") or os.path.join(_HERE, "libmoe.so")

MOE_AFFINE, MOE_SYMMETRIC, MOE_DENSE = 0, 1, 2
MOE_BF16, MOE_FP16 = 0, 1


class MoeError(RuntimeError):
    pass


class QFormatC(C.Structure):
    _fields_ = [("bits", C.c_int32), ("group", C.c_int32), ("mode", C.c_int32),
                ("scale_dtype", C.c_int32)]


class LayerDescC(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("n_experts", C.c_int32), ("top_k", C.c_int32),
                ("inter", C.c_int32), ("shared_inter", C.c_int32), ("act_dtype", C.c_int32),
                ("router", QFormatC), ("gate_row", QFormatC), ("routed", QFormatC),
                ("shared", QFormatC)]


class QTensorC(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("biases", C.c_void_p)]


class LayerSrcC(C.Structure):
    _fields_ = [(n, QTensorC) for n in
                ("router", "gate_row", "gate", "up", "down", "sh_gate", "sh_up", "sh_down")]


class MatOffC(C.Structure):
    _fields_ = [("codes", C.c_uint64), ("scales", C.c_uint64)]


class LayerC(C.Structure):
    _fields_ = [("d", LayerDescC), ("dev", C.c_void_p), ("bytes", C.c_uint64),
                ("router_off", C.c_uint64), ("router_scale_off", C.c_uint64),
                ("gate_row_off", C.c_uint64), ("gate_row_scale_off", C.c_uint64),
                ("experts_off", C.c_uint64), ("expert_stride", C.c_uint64),
                ("gu", MatOffC), ("dn", MatOffC), ("shared_off", C.c_uint64),
                ("sh_gu", MatOffC), ("sh_dn", MatOffC), ("flags", C.c_uint32)]


class TapsC(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("gu", C.c_void_p), ("h", C.c_void_p), ("e", C.c_void_p),
                ("kernel_events", C.c_void_p * 8), ("route_wait_limit", C.c_int32)]


class GluC(C.Structure):
    _fields_ = [("rows", C.c_int32), ("hidden", C.c_int32), ("inter", C.c_int32), ("dtype", C.c_int32),
                ("act", C.c_int32), ("w_gate", C.c_void_p), ("w_up", C.c_void_p), ("ldw_gate", C.c_int64),
                ("ldw_up", C.c_int64), ("s_gate", C.c_void_p), ("s_up", C.c_void_p), ("x", C.c_void_p),
                ("ldx", C.c_int64), ("s_x", C.c_void_p)]


class LinearC(C.Structure):
    # `in` is a keyword of the language: the member is in_
    _fields_ = [("rows", C.c_int32), ("in_", C.c_int32), ("out", C.c_int32), ("dtype", C.c_int32),
                ("w", C.c_void_p), ("ldw", C.c_int64), ("s_w", C.c_void_p), ("bias", C.c_void_p),
                ("x", C.c_void_p), ("ldx", C.c_int64), ("s_x", C.c_void_p)]


class NormC(C.Structure):
    _fields_ = [("rows", C.c_int32), ("hidden", C.c_int32), ("dtype", C.c_int32), ("x_dtype", C.c_int32),
                ("w_dtype", C.c_int32), ("unit_offset", C.c_int32), ("eps", C.c_float), ("x", C.c_void_p),
                ("ldx", C.c_int64), ("residual", C.c_void_p), ("ldresidual", C.c_int64), ("w", C.c_void_p)]


class LoraC(C.Structure):
    _fields_ = [("rows", C.c_int32), ("in_", C.c_int32), ("out", C.c_int32), ("rank", C.c_int32),
                ("adapters", C.c_int32), ("dtype", C.c_int32), ("x", C.c_void_p), ("ldx", C.c_int64),
                ("a", C.c_void_p), ("lda", C.c_int64), ("stride_a", C.c_int64), ("b", C.c_void_p),
                ("ldb", C.c_int64), ("stride_b", C.c_int64), ("scale", C.c_void_p), ("ids", C.c_void_p)]


EXPORTS = ["moe_pack_size", "moe_pack_layer_host", "moe_layer_bind", "moe_pack_layer",
           "moe_workspace_size", "moe_route", "moe_experts_decode", "moe_experts_grouped",
           "moe_forward_windows", "moe_forward_windows_noalloc", "moe_route_failures",
           "moe_forward_exact", "moe_glu_workspace_size", "moe_glu_forward", "moe_glu_backward", "moe_glu_i8",
           "moe_quant_rows", "moe_linear_i8_workspace_size", "moe_linear_i8",
           "moe_norm_forward", "moe_norm_i8", "moe_norm_backward_workspace_size", "moe_norm_backward",
           "moe_balance_workspace_size", "moe_balance_forward", "moe_balance_backward",
           "moe_lora_workspace_size", "moe_lora_forward", "moe_lora_backward", "moe_status_string", "moe_last_error", "moe_version"]

MOE_WS_DECODE, MOE_WS_GROUPED, MOE_WS_EXACT = 0, 1, 2
MOE_FP32 = 16
MOE_GLU_FORWARD, MOE_GLU_BACKWARD, MOE_GLU_I8 = 0, 1, 2
MOE_LORA_FORWARD, MOE_LORA_BACKWARD = 0, 1
ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}

_lib = None


def lib() -> C.CDLL:
    """Loads libmoe.so (built in-tree by build()); raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise MoeError(f"{LIB_PATH} is missing: build it first "
                       "(python -m quantized_routed_expert_fp32_amd.csrc.build)")
    L = C.CDLL(LIB_PATH)
    vp, i32, u64 = C.c_void_p, C.c_int32, C.c_uint64
    L.moe_pack_size.argtypes = [C.POINTER(LayerDescC), C.POINTER(u64)]
    L.moe_pack_layer_host.argtypes = [C.POINTER(LayerDescC), C.POINTER(LayerSrcC), vp, u64,
                                      C.POINTER(LayerC)]
    L.moe_layer_bind.argtypes = [C.POINTER(LayerC), vp]
    L.moe_pack_layer.argtypes = [C.POINTER(LayerDescC), C.POINTER(LayerSrcC), vp, u64, vp,
                                 C.POINTER(LayerC)]
    L.moe_workspace_size.argtypes = [C.POINTER(LayerDescC), i32, i32, C.POINTER(u64)]
    L.moe_route.argtypes = [C.POINTER(LayerC), vp, i32, vp, vp, vp, vp, vp, u64, C.POINTER(TapsC),
                            vp]
    L.moe_experts_decode.argtypes = [C.POINTER(LayerC), vp, i32, vp, vp, vp, vp, vp, u64,
                                     C.POINTER(TapsC), vp]
    L.moe_experts_grouped.argtypes = L.moe_experts_decode.argtypes
    L.moe_forward_windows.argtypes = [C.POINTER(LayerC), vp, i32, vp, vp, vp, vp, vp, vp, u64, vp]
    L.moe_route_failures.argtypes = [vp, u64, i32, C.POINTER(C.c_uint32), vp]
    L.moe_forward_windows_noalloc.argtypes = [C.POINTER(LayerC), vp, i32, vp, vp, vp, vp, vp, vp]
    L.moe_forward_exact.argtypes = [C.POINTER(LayerC), vp, i32, vp, vp, vp, vp, vp, vp, u64,
                                    C.POINTER(TapsC), vp]
    i64 = C.c_int64
    L.moe_glu_workspace_size.argtypes = [C.POINTER(GluC), i32, C.POINTER(u64)]
    L.moe_glu_forward.argtypes = [C.POINTER(GluC), vp, i64, vp, vp, u64, vp]
    L.moe_glu_backward.argtypes = [C.POINTER(GluC), vp, vp, i64, vp, i64, vp, vp, vp, u64, vp]
    L.moe_glu_i8.argtypes = [C.POINTER(GluC), vp, i64, vp, u64, vp]
    L.moe_quant_rows.argtypes = [vp, i32, i32, i32, i64, vp, i64, vp, vp]
    L.moe_linear_i8_workspace_size.argtypes = [C.POINTER(LinearC), C.POINTER(u64)]
    L.moe_linear_i8.argtypes = [C.POINTER(LinearC), vp, i64, vp, u64, vp]
    L.moe_norm_forward.argtypes = [C.POINTER(NormC), vp, i64, vp, i64, vp, vp]
    L.moe_norm_i8.argtypes = [C.POINTER(NormC), vp, i64, vp, i64, vp, vp, i64, vp]
    L.moe_norm_backward_workspace_size.argtypes = [C.POINTER(NormC), C.POINTER(u64)]
    L.moe_norm_backward.argtypes = [C.POINTER(NormC), vp, vp, i64, vp, i64, vp, i64, vp, vp, u64, vp]
    L.moe_balance_workspace_size.argtypes = [i32, i32, C.POINTER(u64)]
    L.moe_balance_forward.argtypes = [vp, i32, i64, vp, vp, i32, i32, i32, vp, vp, vp, u64, vp]
    L.moe_balance_backward.argtypes = [vp, vp, i32, i64, vp, i32, i32, i32, vp, vp, i64, vp]
    L.moe_lora_workspace_size.argtypes = [C.POINTER(LoraC), i32, C.POINTER(u64)]
    L.moe_lora_forward.argtypes = [C.POINTER(LoraC), vp, i64, vp, i64, vp, vp, u64, vp]
    L.moe_lora_backward.argtypes = [C.POINTER(LoraC), vp, i64, vp, vp, i64, vp, i64, vp, vp, vp, u64, vp]
    for f in ("moe_glu_workspace_size", "moe_glu_forward", "moe_glu_backward", "moe_glu_i8", "moe_quant_rows",
              "moe_linear_i8_workspace_size", "moe_linear_i8", "moe_norm_forward", "moe_norm_i8",
              "moe_norm_backward_workspace_size", "moe_norm_backward", "moe_balance_workspace_size",
              "moe_balance_forward", "moe_balance_backward", "moe_lora_workspace_size", "moe_lora_forward",
              "moe_lora_backward"):
        getattr(L, f).restype = C.c_int
    for f in ("moe_pack_size", "moe_pack_layer_host", "moe_layer_bind", "moe_pack_layer",
              "moe_workspace_size", "moe_route", "moe_experts_decode", "moe_experts_grouped",
              "moe_forward_windows", "moe_forward_windows_noalloc", "moe_route_failures",
              "moe_forward_exact"):
        getattr(L, f).restype = C.c_int
    L.moe_status_string.argtypes = [C.c_int]
    L.moe_status_string.restype = C.c_char_p
    L.moe_last_error.restype = C.c_char_p
    L.moe_version.restype = C.c_char_p
    _lib = L
    return L


def _check(st: int, what: str):
    if st != 0:
        L = lib()
        raise MoeError(f"{what}: {L.moe_status_string(st).decode()}: "
                       f"{L.moe_last_error().decode()}")


# ---------------------------------------------------------------- descriptors
def qformat(bits: int, group: int, mode: int, scale_dtype: int) -> QFormatC:
    return QFormatC(bits, group, mode, scale_dtype)


def layer_desc(hidden, n_experts, top_k, inter, shared_inter, act_dtype,
               router, gate_row, routed, shared) -> LayerDescC:
    """Formats are (bits, group, mode, scale_dtype) tuples or QFormatC."""
    f = lambda q: q if isinstance(q, QFormatC) else QFormatC(*q)
    return LayerDescC(hidden, n_experts, top_k, inter, shared_inter, act_dtype,
                      f(router), f(gate_row), f(routed), f(shared))


def pack_size(desc: LayerDescC) -> int:
    n = C.c_uint64()
    _check(lib().moe_pack_size(C.byref(desc), C.byref(n)), "moe_pack_size")
    return n.value


def _qt(codes, scales, biases, keep):
    arrs = [np.ascontiguousarray(a) if a is not None else None for a in (codes, scales, biases)]
    keep.extend(a for a in arrs if a is not None)
    return QTensorC(*(a.ctypes.data if a is not None else None for a in arrs))


def layer_src(tensors: dict, keep: list) -> LayerSrcC:
    """tensors: name -> (codes, scales, biases) numpy arrays in the canonical layout."""
    return LayerSrcC(*(_qt(*tensors[n], keep) for n in
                       ("router", "gate_row", "gate", "up", "down", "sh_gate", "sh_up", "sh_down")))


def pack_layer_host(desc: LayerDescC, tensors: dict):
    """Host repack into the kernel layout: (uint8 array, LayerC with dev = NULL)."""
    keep = []
    src = layer_src(tensors, keep)
    nbytes = pack_size(desc)
    buf = np.zeros(nbytes, np.uint8)
    out = LayerC()
    _check(lib().moe_pack_layer_host(C.byref(desc), C.byref(src), buf.ctypes.data, nbytes,
                                     C.byref(out)), "moe_pack_layer_host")
    return buf, out


def _stream_ptr(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


@dataclass
class Layer:
    """A packed layer on the device: the LayerC struct and the tensor that owns the bytes."""
    c: LayerC
    buf: object       # torch.uint8 device tensor
    desc: LayerDescC

    @property
    def hidden(self):
        return self.desc.hidden

    @property
    def top_k(self):
        return self.desc.top_k

    @property
    def n_experts(self):
        return self.desc.n_experts


def pack_layer(desc: LayerDescC, tensors: dict, device="cuda", stream=None) -> Layer:
    """Repack on the host and copy to a new device buffer (moe_pack_layer)."""
    import torch
    keep = []
    src = layer_src(tensors, keep)
    nbytes = pack_size(desc)
    buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    base = buf.data_ptr()
    pad = (-base) % 256
    out = LayerC()
    _check(lib().moe_pack_layer(C.byref(desc), C.byref(src), C.c_void_p(base + pad), nbytes,
                                _stream_ptr(stream), C.byref(out)), "moe_pack_layer")
    return Layer(out, buf, desc)


def workspace_size(desc: LayerDescC, rows: int, grouped) -> int:
    """grouped: False / True (decode / grouped form) or one of MOE_WS_*."""
    n = C.c_uint64()
    _check(lib().moe_workspace_size(C.byref(desc), rows, int(grouped), C.byref(n)),
           "moe_workspace_size")
    return n.value


def new_workspace(layer: "Layer", rows: int, grouped, device="cuda", stream=None):
    """A zero-filled workspace for `rows` rows (route + experts of one layer),
    allocated and cleared on `stream` (default: the current stream), so that
    calls enqueued on that stream find it cleared."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    with torch.cuda.stream(s):
        return torch.zeros(workspace_size(layer.desc, rows, grouped), dtype=torch.uint8, device=device)


def route_failures(ws, clear=True, stream=None) -> int:
    """moe_route_failures: rows whose decode-router hand-off missed the wait
    bound since the count was last cleared (synchronises `stream`)."""
    n = C.c_uint32()
    _check(lib().moe_route_failures(_ptr(ws), ws.numel() * ws.element_size(), int(clear), C.byref(n),
                                    _stream_ptr(stream)), "moe_route_failures")
    return n.value


def _on(stream):
    """Context in which outputs of a call on `stream` are allocated."""
    import torch
    return torch.cuda.stream(stream) if stream is not None else _nullctx()


class _nullctx:
    def __enter__(self):
        return None

    def __exit__(self, *a):
        return False


def _taps(taps: Optional[dict]):
    """taps: dict of optional device tensors logits/gu/h/e and an optional
    list "events" of torch.cuda.Event (or None) bracketing each kernel."""
    if not taps:
        return None
    t = TapsC()
    for k in ("logits", "gu", "h", "e"):
        v = taps.get(k)
        setattr(t, k, v.data_ptr() if v is not None else None)
    for i, ev in enumerate(taps.get("events") or []):
        t.kernel_events[i] = ev.cuda_event if ev is not None else None
    t.route_wait_limit = int(taps.get("route_wait_limit", 0))
    return C.byref(t)


def _ptr(t):
    return C.c_void_p(t.data_ptr()) if t is not None else None


def route(layer: Layer, x, logit_bias=None, taps=None, out=None, ws=None, stream=None):
    """moe_route: returns (ids int32 [R,k], p fp32 [R,k], shared_gate fp32 [R])."""
    import torch
    R = x.shape[0]
    k = layer.desc.top_k
    with _on(stream):
        if out is None:
            ids = torch.empty((R, k), dtype=torch.int32, device=x.device)
            p = torch.empty((R, k), dtype=torch.float32, device=x.device)
            sg = torch.empty((R,), dtype=torch.float32, device=x.device)
        else:
            ids, p, sg = out
    if ws is None:
        ws = new_workspace(layer, R, R > 16, x.device, stream)
    _check(lib().moe_route(C.byref(layer.c), _ptr(x), R, _ptr(logit_bias), _ptr(ids), _ptr(p),
                           _ptr(sg), _ptr(ws), ws.numel() * ws.element_size(), _taps(taps),
                           _stream_ptr(stream)), "moe_route")
    return ids, p, sg


def experts(layer: Layer, x, ids, p, sg, grouped: bool, ws=None, taps=None, y=None,
            stream=None):
    """moe_experts_decode (grouped=False) or moe_experts_grouped: returns y fp32 [R,H]."""
    import torch
    R = x.shape[0]
    with _on(stream):
        if y is None:
            y = torch.empty((R, layer.desc.hidden), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = new_workspace(layer, R, grouped, x.device, stream)
    fn = lib().moe_experts_grouped if grouped else lib().moe_experts_decode
    _check(fn(C.byref(layer.c), _ptr(x), R, _ptr(ids), _ptr(p), _ptr(sg), _ptr(y), _ptr(ws),
              ws.numel() * ws.element_size(), _taps(taps), _stream_ptr(stream)),
           "moe_experts_grouped" if grouped else "moe_experts_decode")
    return y


def forward_windows(layer: Layer, x, logit_bias=None, ws=None, out=None, y=None, stream=None):
    """moe_forward_windows: route + decode experts in windows of 16 rows;
    returns (ids, p, shared_gate, y), each row bit-identical to its one-row step."""
    import torch
    R = x.shape[0]
    k = layer.desc.top_k
    with _on(stream):
        if out is None:
            ids = torch.empty((R, k), dtype=torch.int32, device=x.device)
            p = torch.empty((R, k), dtype=torch.float32, device=x.device)
            sg = torch.empty((R,), dtype=torch.float32, device=x.device)
        else:
            ids, p, sg = out
        if y is None:
            y = torch.empty((R, layer.desc.hidden), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = new_workspace(layer, min(R, 16), False, x.device, stream)
    _check(lib().moe_forward_windows(C.byref(layer.c), _ptr(x), R, _ptr(logit_bias), _ptr(ids), _ptr(p),
                                     _ptr(sg), _ptr(y), _ptr(ws), ws.numel() * ws.element_size(),
                                     _stream_ptr(stream)), "moe_forward_windows")
    return ids, p, sg, y


def forward_exact(layer: Layer, x, logit_bias=None, ws=None, out=None, y=None, taps=None, stream=None):
    """moe_forward_exact: the chunk with the decode step's bits for every row
    (sorted into expert blocks); returns (ids, p, shared_gate, y)."""
    import torch
    R = x.shape[0]
    k = layer.desc.top_k
    with _on(stream):
        if out is None:
            ids = torch.empty((R, k), dtype=torch.int32, device=x.device)
            p = torch.empty((R, k), dtype=torch.float32, device=x.device)
            sg = torch.empty((R,), dtype=torch.float32, device=x.device)
        else:
            ids, p, sg = out
        if y is None:
            y = torch.empty((R, layer.desc.hidden), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = new_workspace(layer, R, MOE_WS_EXACT, x.device, stream)
    _check(lib().moe_forward_exact(C.byref(layer.c), _ptr(x), R, _ptr(logit_bias), _ptr(ids), _ptr(p),
                                   _ptr(sg), _ptr(y), _ptr(ws), ws.numel() * ws.element_size(), _taps(taps),
                                   _stream_ptr(stream)), "moe_forward_exact")
    return ids, p, sg, y


def forward_windows_noalloc(layer: Layer, x, logit_bias=None, out=None, y=None, stream=None):
    """moe_forward_windows_noalloc: as forward_windows, with the library's
    fixed device array as the workspace (the call allocates no device
    memory); returns (ids, p, shared_gate, y)."""
    import torch
    R = x.shape[0]
    k = layer.desc.top_k
    with _on(stream):
        if out is None:
            ids = torch.empty((R, k), dtype=torch.int32, device=x.device)
            p = torch.empty((R, k), dtype=torch.float32, device=x.device)
            sg = torch.empty((R,), dtype=torch.float32, device=x.device)
        else:
            ids, p, sg = out
        if y is None:
            y = torch.empty((R, layer.desc.hidden), dtype=torch.float32, device=x.device)
    _check(lib().moe_forward_windows_noalloc(C.byref(layer.c), _ptr(x), R, _ptr(logit_bias), _ptr(ids),
                                             _ptr(p), _ptr(sg), _ptr(y), _stream_ptr(stream)),
           "moe_forward_windows_noalloc")
    return ids, p, sg, y


def experts_decode(layer, x, ids, p, sg, **kw):
    return experts(layer, x, ids, p, sg, False, **kw)


def experts_grouped(layer, x, ids, p, sg, **kw):
    return experts(layer, x, ids, p, sg, True, **kw)


# ------------------------------------------------- dense feed-forward operators
# These calls are short (a decode step's kernel runs for a few microseconds),
# so their checks touch each tensor attribute once and enter a device or
# stream context only where the current one differs.
def _rows2d(t, name, dtype, shape=None, dev=None):
    """Checks a 2-D operand whose rows are contiguous (any row stride); its row
    stride in elements (of a single row: the row length)."""
    if t.dim() != 2:
        raise MoeError(f"{name}: {t.dim()}-D tensor, needs 2 dimensions")
    if t.dtype is not dtype:
        raise MoeError(f"{name}: dtype {t.dtype} is not {dtype}")
    rows, cols = t.shape
    if (rows | cols) >> 31:      # the argument blocks would cut it to 32 bits
        raise MoeError(f"{name}: shape {(rows, cols)}, needs sizes below 2^31")
    if shape is not None and (rows != shape[0] or cols != shape[1]):
        raise MoeError(f"{name}: shape {(rows, cols)}, needs {tuple(shape)}")
    _on_device(t, name, dev)
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise MoeError(f"{name}: the elements of a row must be contiguous (strides {(ld, one)})")
    return ld if rows > 1 else cols


def _on_device(t, name, dev):
    """Checks that t is in device memory, of device `dev` where one is given; its device index."""
    if not t.is_cuda:
        raise MoeError(f"{name}: on {t.device}, needs device memory")
    d = t.get_device()
    if dev is not None and d != dev:
        raise MoeError(f"{name}: on cuda:{d}, x is on cuda:{dev}")
    return d


def _flat(t, name, n, dtype, dev):
    """Checks a contiguous vector of n elements; its address."""
    if t is None:
        return None
    if t.dtype is not dtype or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise MoeError(f"{name}: {t.dtype} of shape {tuple(t.shape)}, needs contiguous {dtype} ({n},)")
    _on_device(t, name, dev)
    return t.data_ptr()


def _half(x, name="x"):
    """MOE_BF16 or MOE_FP16 of a 16-bit operand."""
    import torch
    if x.dtype is torch.bfloat16:
        return MOE_BF16
    if x.dtype is torch.float16:
        return MOE_FP16
    raise MoeError(f"{name}: dtype {x.dtype} is not torch.bfloat16 or torch.float16")


def _no_history(fn, instead, names, *operands):
    """Refuses operands that require a gradient where one would be recorded: the
    result has no history, and a backward pass would leave them out without a word."""
    for t in operands:
        if t is not None and t.requires_grad:
            break
    else:
        return
    import torch
    if torch.is_grad_enabled():
        name = names.split()[[t is not None and t.requires_grad for t in operands].index(True)]
        raise MoeError(f"{fn}: {name} requires a gradient, which this call does not record: {instead}"
                       "call it under torch.no_grad()")


_forward_ad = None


def _no_tangent(fn, names, *operands):
    """Refuses operands that carry a tangent of forward-mode differentiation, which the
    result would lack without a word (torch.no_grad() leaves that mode on)."""
    global _forward_ad
    if _forward_ad is None:                 # (kept: an import statement costs a call 0.7 us)
        from torch.autograd import forward_ad as _forward_ad
    if getattr(_forward_ad, "_current_level", 0) < 0:      # outside every dual_level
        return
    for name, t in zip(names.split(), operands):
        if t is not None and _forward_ad.unpack_dual(t).tangent is not None:
            raise MoeError(f"{fn}: {name} carries a tangent of forward-mode differentiation, which this call does "
                           "not compute: pass forward_ad.unpack_dual(..).primal")


def _act_code(act):
    if act not in ACTIVATIONS:
        raise MoeError(f"act: {act!r} is not one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[act]


def _call_ctx(dev, stream):
    """The context of a call on device `dev`: outputs and the workspace are
    allocated on the stream that uses them, with the device current. None
    where the current ones already are."""
    import torch
    if stream is not None:
        if stream.device.index != dev:
            raise MoeError(f"stream: on {stream.device}, x is on cuda:{dev}")
        return torch.cuda.stream(stream)
    return None if torch.cuda.current_device() == dev else torch.cuda.device(dev)


def _raw_stream(dev, stream):
    import torch
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _workspace(n, ws, dev):
    """(address, bytes, owner) of the workspace of a call that needs n bytes."""
    import torch
    if ws is None:
        if not n:
            return None, 0, None
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        return ws.data_ptr(), n, ws
    if not ws.is_contiguous():
        raise MoeError("ws: needs contiguous memory")
    _on_device(ws, "ws", dev)
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def _glu_args(x, w_gate, w_up, act, s_gate=None, s_up=None, x_scale=None, out_dtype=None):
    """(argument block, output dtype, device index) of a gated-block call."""
    import torch
    i8 = s_gate is not None
    if x_scale is None:
        dt = x.dtype
        code = _half(x)
        ldx = _rows2d(x, "x", dt)
        if out_dtype is not None and out_dtype is not dt:
            raise MoeError(f"out_dtype: {out_dtype} with x of {dt} (it is a choice for int8 x only)")
    else:
        dt = torch.bfloat16 if out_dtype is None else out_dtype
        if dt not in (torch.bfloat16, torch.float16):
            raise MoeError(f"out_dtype: {dt} is not torch.bfloat16 or torch.float16")
        code = MOE_BF16 if dt is torch.bfloat16 else MOE_FP16
        ldx = _rows2d(x, "x", torch.int8)
    dev = x.get_device()
    wt = torch.int8 if i8 else dt
    ldg = _rows2d(w_gate, "w_gate", wt, None, dev)
    R, K = x.shape
    I, H = w_gate.shape
    if K != H:
        raise MoeError(f"x: rows of {K} elements, w_gate has {H} columns")
    ldu = _rows2d(w_up, "w_up", wt, (I, H), dev)
    f32 = torch.float32
    a = GluC(R, H, I, code, _act_code(act), w_gate.data_ptr(), w_up.data_ptr(), ldg, ldu,
             _flat(s_gate, "s_gate", I, f32, dev), _flat(s_up, "s_up", I, f32, dev), x.data_ptr(), ldx,
             _flat(x_scale, "x_scale", R, f32, dev))
    return a, dt, dev


def _glu_need(a, kind):
    n = C.c_uint64()
    st = lib().moe_glu_workspace_size(C.byref(a), kind, C.byref(n))
    if st:
        _check(st, "moe_glu_workspace_size")
    return n.value


def glu_workspace_size(x, w_gate, w_up, kind=MOE_GLU_FORWARD, s_gate=None, s_up=None, x_scale=None) -> int:
    """moe_glu_workspace_size of a call on these tensors, in bytes."""
    return _glu_need(_glu_args(x, w_gate, w_up, "silu", s_gate, s_up, x_scale)[0], kind)


def glu_forward(x, w_gate, w_up, act="silu", save=False, h=None, gu=None, ws=None, stream=None):
    """moe_glu_forward: h = act(x w_gate^T) * (x w_up^T), [rows, inter] of x's
    dtype (bf16 or fp16); with save=True (h, gu), gu fp32 [rows, 2, inter] being what
    glu_backward takes. h has no autograd history: without save (or gu), operands
    that require a gradient are refused where grad mode is on."""
    _no_tangent("glu_forward", "x w_gate w_up", x, w_gate, w_up)
    if not save and gu is None:
        _no_history("glu_forward", "take save=True and glu_backward, or ", "x w_gate w_up", x, w_gate, w_up)
    a, dt, dev = _glu_args(x, w_gate, w_up, act)
    ctx = _call_ctx(dev, stream)
    if ctx is None:
        return _glu_forward(a, dt, dev, save, h, gu, ws, stream)
    with ctx:
        return _glu_forward(a, dt, dev, save, h, gu, ws, stream)


def _glu_forward(a, dt, dev, save, h, gu, ws, stream):
    import torch
    R, I = a.rows, a.inter
    n = _glu_need(a, MOE_GLU_FORWARD)
    if h is None:
        h, ldh = torch.empty((R, I), dtype=dt, device=dev), I
    else:
        ldh = _rows2d(h, "h", dt, (R, I), dev)
    gp = None
    if gu is not None:
        gp = _gu_ok(gu, R, I, dev)
    elif save:
        gu = torch.empty((R, 2, I), dtype=torch.float32, device=dev)
        gp = gu.data_ptr()
    wp, wn, ws = _workspace(n, ws, dev)
    st = lib().moe_glu_forward(C.byref(a), h.data_ptr(), ldh, gp, wp, wn, _raw_stream(dev, stream))
    if st:
        _check(st, "moe_glu_forward")
    return (h, gu) if gu is not None else h


def _gu_ok(gu, R, I, dev):
    import torch
    if gu.dtype is not torch.float32 or tuple(gu.shape) != (R, 2, I) or not gu.is_contiguous():
        raise MoeError(f"gu: {gu.dtype} of shape {tuple(gu.shape)}, needs contiguous torch.float32 ({R}, 2, {I})")
    _on_device(gu, "gu", dev)
    return gu.data_ptr()


def glu_backward(dh, x, w_gate, w_up, gu, act="silu", need_dx=True, need_dw=True, dx=None, dw_gate=None,
                 dw_up=None, ws=None, stream=None):
    """moe_glu_backward: (dx, dw_gate, dw_up) of glu_forward(..., save=True) from
    dh and its gu; None in the place of a gradient that is not needed. Gradients
    of these gradients are not computed: a dh that requires one is refused."""
    _no_tangent("glu_backward", "dh x w_gate w_up gu", dh, x, w_gate, w_up, gu)
    _no_history("glu_backward", "", "dh", dh)
    a, dt, dev = _glu_args(x, w_gate, w_up, act)
    if not need_dx and not need_dw:
        raise MoeError("glu_backward: neither need_dx nor need_dw")
    lddh = _rows2d(dh, "dh", dt, (a.rows, a.inter), dev)
    gp = _gu_ok(gu, a.rows, a.inter, dev)
    outs = (dx if need_dx else None, dw_gate if need_dw else None, dw_up if need_dw else None)
    ctx = _call_ctx(dev, stream)
    if ctx is None:
        return _glu_backward(a, dt, dev, dh.data_ptr(), lddh, gp, need_dx, need_dw, outs, ws, stream)
    with ctx:
        return _glu_backward(a, dt, dev, dh.data_ptr(), lddh, gp, need_dx, need_dw, outs, ws, stream)


def _glu_backward(a, dt, dev, dhp, lddh, gp, need_dx, need_dw, outs, ws, stream):
    import torch
    R, H, I = a.rows, a.hidden, a.inter
    n = _glu_need(a, MOE_GLU_BACKWARD)
    dx, dwg, dwu = outs
    lddx = H
    if need_dx:
        if dx is None:
            dx = torch.empty((R, H), dtype=dt, device=dev)
        else:
            lddx = _rows2d(dx, "dx", dt, (R, H), dev)
    if need_dw:
        if dwg is None:
            dwg = torch.empty((I, H), dtype=dt, device=dev)
        elif _rows2d(dwg, "dw_gate", dt, (I, H), dev) != H:
            raise MoeError("dw_gate: needs contiguous memory")
        if dwu is None:
            dwu = torch.empty((I, H), dtype=dt, device=dev)
        elif _rows2d(dwu, "dw_up", dt, (I, H), dev) != H:
            raise MoeError("dw_up: needs contiguous memory")
    wp, wn, ws = _workspace(n, ws, dev)
    st = lib().moe_glu_backward(C.byref(a), gp, dhp, lddh, dx.data_ptr() if need_dx else None, lddx,
                                dwg.data_ptr() if need_dw else None, dwu.data_ptr() if need_dw else None, wp, wn,
                                _raw_stream(dev, stream))
    if st:
        _check(st, "moe_glu_backward")
    return dx, dwg, dwu


def glu_i8(x, w_gate, s_gate, w_up, s_up, act="silu", x_scale=None, out_dtype=None, h=None, ws=None, stream=None):
    """moe_glu_i8: the gated block on int8 weights [inter, hidden] with fp32
    channel scales [inter]; x in bf16/fp16 (quantised a token inside the call),
    or int8 with x_scale [rows] (then out_dtype is h's type, bf16 by default). No
    gradients: operands that require one are refused where grad mode is on."""
    _no_tangent("glu_i8", "x s_gate s_up x_scale", x, s_gate, s_up, x_scale)
    _no_history("glu_i8", "", "x s_gate s_up x_scale", x, s_gate, s_up, x_scale)
    if s_gate is None or s_up is None:
        raise MoeError("s_gate, s_up: needed with int8 weights")
    a, dt, dev = _glu_args(x, w_gate, w_up, act, s_gate, s_up, x_scale, out_dtype)
    ctx = _call_ctx(dev, stream)
    if ctx is None:
        return _glu_i8(a, dt, dev, h, ws, stream)
    with ctx:
        return _glu_i8(a, dt, dev, h, ws, stream)


def _glu_i8(a, dt, dev, h, ws, stream):
    import torch
    n = _glu_need(a, MOE_GLU_I8)
    if h is None:
        h, ldh = torch.empty((a.rows, a.inter), dtype=dt, device=dev), a.inter
    else:
        ldh = _rows2d(h, "h", dt, (a.rows, a.inter), dev)
    wp, wn, ws = _workspace(n, ws, dev)
    st = lib().moe_glu_i8(C.byref(a), h.data_ptr(), ldh, wp, wn, _raw_stream(dev, stream))
    if st:
        _check(st, "moe_glu_i8")
    return h


def quant_rows(x, q=None, scale=None, stream=None):
    """moe_quant_rows: rows of x (bf16, fp16 or fp32) as (int8 [rows, cols],
    fp32 scale [rows]); of a weight matrix [out, in] the rows are its channels.
    Neither has a gradient (rounding has none)."""
    import torch
    code = MOE_FP32 if x.dtype is torch.float32 else _half(x)
    ldx = _rows2d(x, "x", x.dtype)
    dev = x.get_device()
    ctx = _call_ctx(dev, stream)
    with ctx if ctx is not None else _nullctx():
        R, K = x.shape
        if q is None:
            q = torch.empty((R, K), dtype=torch.int8, device=dev)
        elif _rows2d(q, "q", torch.int8, (R, K), dev) != K:
            raise MoeError("q: needs contiguous memory")
        if scale is None:
            scale = torch.empty((R,), dtype=torch.float32, device=dev)
        sp = _flat(scale, "scale", R, torch.float32, dev)
        _check(lib().moe_quant_rows(x.data_ptr(), code, R, K, ldx, q.data_ptr(), K, sp, _raw_stream(dev, stream)),
               "moe_quant_rows")
    return q, scale


def _linear_args(x, w, s_w, bias, x_scale, out_dtype):
    """(argument block, output dtype, device index) of a linear_i8 call."""
    import torch
    f32 = torch.float32
    if x_scale is None:
        dt = x.dtype
        code = _half(x)
        ldx = _rows2d(x, "x", dt)
        if out_dtype is not None and out_dtype is not dt:
            raise MoeError(f"out_dtype: {out_dtype} with x of {dt} (it is a choice for int8 x only)")
    else:
        dt = torch.bfloat16 if out_dtype is None else out_dtype
        if dt not in (torch.bfloat16, torch.float16):
            raise MoeError(f"out_dtype: {dt} is not torch.bfloat16 or torch.float16")
        code = MOE_BF16 if dt is torch.bfloat16 else MOE_FP16
        ldx = _rows2d(x, "x", torch.int8)
    dev = x.get_device()
    ldw = _rows2d(w, "w", torch.int8, None, dev)
    N, K = w.shape
    R, Kx = x.shape
    if Kx != K:
        raise MoeError(f"x: rows of {Kx} elements, w has {K} columns")
    if s_w is None:
        raise MoeError("s_w: needed with int8 weights")
    a = LinearC(R, K, N, code, w.data_ptr(), ldw, _flat(s_w, "s_w", N, f32, dev), _flat(bias, "bias", N, f32, dev),
                x.data_ptr(), ldx, _flat(x_scale, "x_scale", R, f32, dev))
    return a, dt, dev


def _linear_need(a):
    n = C.c_uint64()
    st = lib().moe_linear_i8_workspace_size(C.byref(a), C.byref(n))
    if st:
        _check(st, "moe_linear_i8_workspace_size")
    return n.value


def linear_i8_workspace_size(x, w, s_w, x_scale=None) -> int:
    """moe_linear_i8_workspace_size of a call on these tensors, in bytes."""
    return _linear_need(_linear_args(x, w, s_w, None, x_scale, None)[0])


def linear_i8(x, w, s_w, bias=None, x_scale=None, out_dtype=None, y=None, ws=None, stream=None):
    """moe_linear_i8: y = x w^T (+ bias) for int8 w [out, in] with fp32 channel
    scales s_w [out]; x in bf16/fp16 (quantised a token inside the call), or
    int8 with x_scale [rows] (then out_dtype is y's type, bf16 by default). No
    gradients: operands that require one are refused where grad mode is on."""
    _no_tangent("linear_i8", "x s_w bias x_scale", x, s_w, bias, x_scale)
    _no_history("linear_i8", "", "x s_w bias x_scale", x, s_w, bias, x_scale)
    a, dt, dev = _linear_args(x, w, s_w, bias, x_scale, out_dtype)
    ctx = _call_ctx(dev, stream)
    if ctx is None:
        return _linear_i8(a, dt, dev, y, ws, stream)
    with ctx:
        return _linear_i8(a, dt, dev, y, ws, stream)


def _linear_i8(a, dt, dev, y, ws, stream):
    import torch
    n = _linear_need(a)
    if y is None:
        y, ldy = torch.empty((a.rows, a.out), dtype=dt, device=dev), a.out
    else:
        ldy = _rows2d(y, "y", dt, (a.rows, a.out), dev)
    wp, wn, ws = _workspace(n, ws, dev)
    st = lib().moe_linear_i8(C.byref(a), y.data_ptr(), ldy, wp, wn, _raw_stream(dev, stream))
    if st:
        _check(st, "moe_linear_i8")
    return y


# ----------------------------------- operators around the feed-forward block
def _in(dev, stream, fn, *args):
    """fn(*args) with device `dev` (and the stream, if one is given) current."""
    ctx = _call_ctx(dev, stream)
    if ctx is None:
        return fn(*args)
    with ctx:
        return fn(*args)


def _like(t, name, dtype, shape, dev):
    """(tensor, row stride) of an output: the caller's, checked, or a new one."""
    import torch
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev), shape[1]
    return t, _rows2d(t, name, dtype, shape, dev)


def _vector(t, name, n, dtype, dev):
    """A contiguous output vector: the caller's, checked, or a new one."""
    import torch
    if t is None:
        return torch.empty((n,), dtype=dtype, device=dev)
    _flat(t, name, n, dtype, dev)
    return t


def _norm_args(x, weight, eps, residual, unit_offset):
    """(argument block, result dtype, device index) of a norm call."""
    import torch
    dt = x.dtype if residual is None else residual.dtype
    code = _half(x) if residual is None else _half(residual, "residual")
    ldx = _rows2d(x, "x", torch.float32 if x.dtype is torch.float32 else dt)
    dev = x.get_device()
    R, H = x.shape
    ldr = 0 if residual is None else _rows2d(residual, "residual", dt, (R, H), dev)
    wt = torch.float32 if weight.dtype is torch.float32 else dt
    a = NormC(R, H, code, code if x.dtype is dt else MOE_FP32, code if wt is dt else MOE_FP32, int(bool(unit_offset)),
              eps, x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr,
              _flat(weight, "weight", H, wt, dev))
    return a, dt, dev


def _total(total, residual, R, H, dt, dev):
    """(tensor, address, row stride) of a call's total; none without a residual."""
    if residual is None:
        if total is not None:
            raise MoeError("total: given without a residual")
        return None, None, 0
    total, ld = _like(total, "total", dt, (R, H), dev)
    return total, total.data_ptr(), ld


def norm_forward(x, weight, eps=1e-6, residual=None, unit_offset=False, save=False, total=None, y=None, rstd=None,
                 stream=None):
    """moe_norm_forward: (y, total, rstd), total = x + residual and y its root-mean-square
    norm times weight (1 + weight with unit_offset). x [rows, hidden] of bf16 or fp16,
    or with a residual of one of them fp32 (what experts() returns); weight of the same
    type or fp32. total is None without a residual (it may be passed as the residual
    itself: then it is updated in place), rstd without save (or rstd); total (or x)
    and rstd are what norm_backward takes. Nothing has autograd history: without
    save, operands that require a gradient are refused where grad mode is on."""
    _no_tangent("norm_forward", "x weight residual", x, weight, residual)
    if not save and rstd is None:
        _no_history("norm_forward", "take save=True and norm_backward, or ", "x weight residual", x, weight, residual)
    a, dt, dev = _norm_args(x, weight, eps, residual, unit_offset)
    return _in(dev, stream, _norm_forward, a, dt, dev, residual, save, total, y, rstd, stream)


def _norm_forward(a, dt, dev, residual, save, total, y, rstd, stream):
    import torch
    R, H = a.rows, a.hidden
    total, tp, ldt = _total(total, residual, R, H, dt, dev)
    y, ldy = _like(y, "y", dt, (R, H), dev)
    if save or rstd is not None:
        rstd = _vector(rstd, "rstd", R, torch.float32, dev)
    st = lib().moe_norm_forward(C.byref(a), tp, ldt, y.data_ptr(), ldy, None if rstd is None else rstd.data_ptr(),
                                _raw_stream(dev, stream))
    if st:
        _check(st, "moe_norm_forward")
    return y, total, rstd


def norm_i8(x, weight, eps=1e-6, residual=None, unit_offset=False, want_y=False, total=None, q=None, scale=None, y=None,
            stream=None):
    """moe_norm_i8: (q, scale, total, y): the norm's result as int8 rows with an fp32
    scale each, what linear_i8 and glu_i8 take as x and x_scale; y is the 16-bit result
    too (with want_y or y, else None), total as in norm_forward. No gradients: operands
    that require one are refused where grad mode is on."""
    _no_tangent("norm_i8", "x weight residual", x, weight, residual)
    _no_history("norm_i8", "", "x weight residual", x, weight, residual)
    a, dt, dev = _norm_args(x, weight, eps, residual, unit_offset)
    return _in(dev, stream, _norm_i8, a, dt, dev, residual, want_y, total, q, scale, y, stream)


def _norm_i8(a, dt, dev, residual, want_y, total, q, scale, y, stream):
    import torch
    R, H = a.rows, a.hidden
    total, tp, ldt = _total(total, residual, R, H, dt, dev)
    q, ldq = _like(q, "q", torch.int8, (R, H), dev)
    scale = _vector(scale, "scale", R, torch.float32, dev)
    ldy = 0
    if want_y or y is not None:
        y, ldy = _like(y, "y", dt, (R, H), dev)
    st = lib().moe_norm_i8(C.byref(a), tp, ldt, q.data_ptr(), ldq, scale.data_ptr(), None if y is None else y.data_ptr(),
                           ldy, _raw_stream(dev, stream))
    if st:
        _check(st, "moe_norm_i8")
    return q, scale, total, y


def norm_backward_workspace_size(x, weight) -> int:
    """moe_norm_backward_workspace_size of a call on these tensors, in bytes."""
    return _norm_need(_norm_args(x, weight, 1e-6, None, False)[0])


def _norm_need(a):
    n = C.c_uint64()
    st = lib().moe_norm_backward_workspace_size(C.byref(a), C.byref(n))
    if st:
        _check(st, "moe_norm_backward_workspace_size")
    return n.value


def norm_backward(dy, total, weight, rstd, dtotal=None, unit_offset=False, need_dx=True, need_dw=True, dx=None, dw=None,
                  ws=None, stream=None):
    """moe_norm_backward: (dx, dw) of norm_forward(..., save=True) from dy, its rstd and
    what it normalised (its total, or x where it had no residual). dtotal is the gradient
    that reaches the total itself; dx is the gradient of x and of the residual alike. None
    in the place of a gradient that is not needed. Gradients of these gradients are not
    computed: a dy or dtotal that requires one is refused."""
    _no_tangent("norm_backward", "dy total weight rstd dtotal", dy, total, weight, rstd, dtotal)
    _no_history("norm_backward", "", "dy dtotal", dy, dtotal)
    if not need_dx and not need_dw:
        raise MoeError("norm_backward: neither need_dx nor need_dw")
    if dtotal is not None and not need_dx:
        raise MoeError("dtotal: given without need_dx, the only gradient that it is part of")
    a, dt, dev = _norm_args(total, weight, 1e-6, None, unit_offset)
    import torch
    R, H = a.rows, a.hidden
    lddy = _rows2d(dy, "dy", dt, (R, H), dev)
    up, ldu = (None, 0) if dtotal is None else (dtotal.data_ptr(), _rows2d(dtotal, "dtotal", dt, (R, H), dev))
    rp = _flat(rstd, "rstd", R, torch.float32, dev)
    if rp is None:
        raise MoeError("rstd: needed (norm_forward with save=True returns it)")
    return _in(dev, stream, _norm_backward, a, dt, dev, rp, dy.data_ptr(), lddy, up, ldu,
               weight.dtype, need_dx, need_dw, dx, dw, ws, stream)


def _norm_backward(a, dt, dev, rp, dyp, lddy, up, ldu, wt, need_dx, need_dw, dx, dw, ws, stream):
    R, H = a.rows, a.hidden
    n = _norm_need(a) if need_dw else 0
    ldx = 0
    if need_dx:
        dx, ldx = _like(dx, "dx", dt, (R, H), dev)
    if need_dw:
        dw = _vector(dw, "dw", H, wt, dev)
    wp, wn, ws = _workspace(n, ws, dev)
    st = lib().moe_norm_backward(C.byref(a), rp, dyp, lddy, up, ldu, dx.data_ptr() if need_dx else None, ldx,
                                 dw.data_ptr() if need_dw else None, wp, wn, _raw_stream(dev, stream))
    if st:
        _check(st, "moe_norm_backward")
    return dx if need_dx else None, dw if need_dw else None


def _balance_args(logits, mask):
    """(dtype code, row stride, mask address, device index) of a balance call."""
    import torch
    code = MOE_FP32 if logits.dtype is torch.float32 else _half(logits, "logits")
    ld = _rows2d(logits, "logits", logits.dtype)
    dev = logits.get_device()
    return code, ld, _flat(mask, "mask", logits.shape[0], torch.bool, dev), dev


def balance_workspace_size(rows, experts) -> int:
    """moe_balance_workspace_size, in bytes."""
    n = C.c_uint64()
    st = lib().moe_balance_workspace_size(rows, experts, C.byref(n))
    if st:
        _check(st, "moe_balance_workspace_size")
    return n.value


def balance_forward(logits, ids, mask=None, save=False, losses=None, counts=None, ws=None, stream=None):
    """moe_balance_forward: (losses, counts) of a router's logits [rows, experts] (fp32,
    bf16 or fp16; any row stride, so route's logits beside the shared gate's are
    logits[:, :experts]) and its picks ids [rows, k] int32, over the rows that mask
    [rows] (bool) keeps. losses fp32 [2]: the balance loss experts sum f_e mean(p_e) and
    the z loss mean(logsumexp^2); counts int32 [experts + 1]: picks of each expert, and
    the rows that count. No autograd history: without save=True (the caller runs
    balance_backward, which takes counts), logits that require a gradient are refused
    where grad mode is on."""
    _no_tangent("balance_forward", "logits", logits)
    if not save:
        _no_history("balance_forward", "take save=True and balance_backward, or ", "logits", logits)
    import torch
    code, ld, mp, dev = _balance_args(logits, mask)
    if _rows2d(ids, "ids", torch.int32, (logits.shape[0], ids.shape[-1]), dev) != ids.shape[1]:
        raise MoeError("ids: needs contiguous memory")
    return _in(dev, stream, _balance_forward, logits, code, ld, ids, mp, dev, losses, counts, ws, stream)


def _balance_forward(logits, code, ld, ids, mp, dev, losses, counts, ws, stream):
    import torch
    (R, E), k = logits.shape, ids.shape[1]
    n = balance_workspace_size(R, E)
    losses = _vector(losses, "losses", 2, torch.float32, dev)
    counts = _vector(counts, "counts", E + 1, torch.int32, dev)
    wp, wn, ws = _workspace(n, ws, dev)
    st = lib().moe_balance_forward(logits.data_ptr(), code, ld, ids.data_ptr(), mp, R, E, k, losses.data_ptr(),
                                   counts.data_ptr(), wp, wn, _raw_stream(dev, stream))
    if st:
        _check(st, "moe_balance_forward")
    return losses, counts


def balance_backward(dlosses, logits, counts, k, mask=None, dlogits=None, stream=None):
    """moe_balance_backward: dlogits [rows, experts] of the logits' type, from dlosses
    fp32 [2] (on the device), the counts of balance_forward and its number of picks k.
    Gradients of this gradient are not computed: dlosses that require one are refused."""
    _no_tangent("balance_backward", "dlosses logits", dlosses, logits)
    _no_history("balance_backward", "", "dlosses", dlosses)
    import torch
    code, ld, mp, dev = _balance_args(logits, mask)
    if dlosses is None or counts is None:
        raise MoeError("dlosses, counts: both needed")
    dp = _flat(dlosses, "dlosses", 2, torch.float32, dev)
    cp = _flat(counts, "counts", logits.shape[1] + 1, torch.int32, dev)
    return _in(dev, stream, _balance_backward, dp, logits, code, ld, mp, dev, cp, k, dlogits, stream)


def _balance_backward(dp, logits, code, ld, mp, dev, cp, k, dlogits, stream):
    R, E = logits.shape
    dlogits, ldd = _like(dlogits, "dlogits", logits.dtype, (R, E), dev)
    st = lib().moe_balance_backward(dp, logits.data_ptr(), code, ld, mp, R, E, k, cp, dlogits.data_ptr(), ldd,
                                    _raw_stream(dev, stream))
    if st:
        _check(st, "moe_balance_backward")
    return dlogits


def _stack3d(t, name, dtype, shape, dev):
    """Checks a stack of matrices whose rows are contiguous; (row, matrix) strides in elements."""
    if t.dim() != 3:
        raise MoeError(f"{name}: {t.dim()}-D tensor, needs 3 dimensions")
    if t.dtype is not dtype:
        raise MoeError(f"{name}: dtype {t.dtype} is not {dtype}")
    if any(n >> 31 for n in t.shape):
        raise MoeError(f"{name}: shape {tuple(t.shape)}, needs sizes below 2^31")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise MoeError(f"{name}: shape {tuple(t.shape)}, needs {tuple(shape)}")
    _on_device(t, name, dev)
    s, ld, one = t.stride()
    n, rows, cols = t.shape
    if one != 1 and cols > 1:
        raise MoeError(f"{name}: the elements of a row must be contiguous (strides {(s, ld, one)})")
    return (ld if rows > 1 else cols), (s if n > 1 else 0)


def _lora_args(x, a, b, ids, scale):
    """(argument block, device index) of an adapter call."""
    import torch
    code, dt = _half(x), x.dtype
    ldx = _rows2d(x, "x", dt)
    dev = x.get_device()
    lda, sta = _stack3d(a, "a", dt, None, dev)
    (n, rank, K), (R, Kx) = a.shape, x.shape
    if Kx != K:
        raise MoeError(f"x: rows of {Kx} elements, a has {K} columns")
    if b.dim() != 3:
        raise MoeError(f"b: {b.dim()}-D tensor, needs 3 dimensions")
    N = b.shape[1]
    ldb, stb = _stack3d(b, "b", dt, (n, N, rank), dev)
    if ids is None or scale is None:
        raise MoeError("ids, scale: both needed")
    c = LoraC(R, K, N, rank, n, code, x.data_ptr(), ldx, a.data_ptr(), lda, sta, b.data_ptr(), ldb, stb,
              _flat(scale, "scale", n, torch.float32, dev), _flat(ids, "ids", R, torch.int32, dev))
    return c, dev


def _lora_need(c, kind):
    n = C.c_uint64()
    st = lib().moe_lora_workspace_size(C.byref(c), kind, C.byref(n))
    if st:
        _check(st, "moe_lora_workspace_size")
    return n.value


def lora_workspace_size(x, a, b, ids, scale, kind=MOE_LORA_FORWARD) -> int:
    """moe_lora_workspace_size of a call on these tensors, in bytes."""
    return _lora_need(_lora_args(x, a, b, ids, scale)[0], kind)


def _lora_t(t, R, rank, dev):
    import torch
    if _rows2d(t, "t", torch.float32, (R, rank), dev) != rank:
        raise MoeError("t: needs contiguous memory")
    return t.data_ptr()


def lora_forward(x, a, b, ids, scale, base=None, save=False, y=None, t=None, ws=None, stream=None):
    """moe_lora_forward: y = base + scale[i] (x a[i]^T) b[i]^T with i = ids[row], [rows, out]
    of x's dtype (bf16 or fp16): low-rank adapters a [adapters, rank, in] and b [adapters,
    out, rank] of many requests beside a shared projection, whose result is base (it may
    be passed as y: then it is updated in place). ids int32 [rows], outside 0..adapters-1:
    no adapter; scale fp32 [adapters]. With save=True (or t) (y, t), t fp32 [rows, rank]
    being what lora_backward takes. No autograd history: without save, operands that
    require a gradient are refused where grad mode is on; scale's is never computed."""
    _no_tangent("lora_forward", "x a b scale base", x, a, b, scale, base)
    if not save and t is None:
        _no_history("lora_forward", "take save=True and lora_backward, or ", "x a b scale base", x, a, b, scale, base)
    else:
        _no_history("lora_forward", "", "scale", scale)
    c, dev = _lora_args(x, a, b, ids, scale)
    return _in(dev, stream, _lora_forward, c, x.dtype, dev, base, save, y, t, ws, stream)


def _lora_forward(c, dt, dev, base, save, y, t, ws, stream):
    import torch
    R, N = c.rows, c.out
    n = _lora_need(c, MOE_LORA_FORWARD)
    bp, ldb = (None, 0) if base is None else (base.data_ptr(), _rows2d(base, "base", dt, (R, N), dev))
    y, ldy = _like(y, "y", dt, (R, N), dev)
    tp = None
    if t is not None:
        tp = _lora_t(t, R, c.rank, dev)
    elif save:
        t = torch.empty((R, c.rank), dtype=torch.float32, device=dev)
        tp = t.data_ptr()
    wp, wn, ws = _workspace(n, ws, dev)
    st = lib().moe_lora_forward(C.byref(c), bp, ldb, y.data_ptr(), ldy, tp, wp, wn, _raw_stream(dev, stream))
    if st:
        _check(st, "moe_lora_forward")
    return (y, t) if t is not None else y


def lora_backward(dy, x, a, b, ids, scale, t=None, dx_base=None, need_dx=True, need_dw=True, dx=None, da=None, db=None,
                  ws=None, stream=None):
    """moe_lora_backward: (dx, da, db) of lora_forward(..., save=True) from dy and its t
    (not read without need_dw). dx_base [rows, in] is added to dx: the gradient through the
    shared projection (it may be passed as dx: then it is updated in place; a dx_base that is
    dy itself only without need_dw, as da and db read dy behind it). The gradient of base
    is dy itself. None in the place of a gradient that is not needed.
    Gradients of these gradients are not computed: a dy or dx_base that requires one
    is refused."""
    _no_tangent("lora_backward", "dy x a b scale t dx_base", dy, x, a, b, scale, t, dx_base)
    _no_history("lora_backward", "", "dy dx_base", dy, dx_base)
    if not need_dx and not need_dw:
        raise MoeError("lora_backward: neither need_dx nor need_dw")
    if dx_base is not None and not need_dx:
        raise MoeError("dx_base: given without need_dx")
    c, dev = _lora_args(x, a, b, ids, scale)
    lddy = _rows2d(dy, "dy", x.dtype, (c.rows, c.out), dev)
    if need_dw and t is None:
        raise MoeError("t: needed for da and db (lora_forward with save=True returns it)")
    tp = _lora_t(t, c.rows, c.rank, dev) if need_dw else None
    return _in(dev, stream, _lora_backward, c, x.dtype, dev, dy.data_ptr(), lddy, tp, dx_base, need_dx, need_dw, dx, da,
               db, ws, stream)


def _lora_backward(c, dt, dev, dyp, lddy, tp, dx_base, need_dx, need_dw, dx, da, db, ws, stream):
    import torch
    R, K, N, n, rank = c.rows, c.in_, c.out, c.adapters, c.rank
    need = _lora_need(c, MOE_LORA_BACKWARD)
    bp, ldbase = (None, 0) if dx_base is None else (dx_base.data_ptr(), _rows2d(dx_base, "dx_base", dt, (R, K), dev))
    ldx = 0
    if need_dx:
        dx, ldx = _like(dx, "dx", dt, (R, K), dev)
    if need_dw:
        da = _stack_out(da, "da", dt, (n, rank, K), dev)
        db = _stack_out(db, "db", dt, (n, N, rank), dev)
    wp, wn, ws = _workspace(need, ws, dev)
    st = lib().moe_lora_backward(C.byref(c), dyp, lddy, tp, bp, ldbase, dx.data_ptr() if need_dx else None, ldx,
                                 da.data_ptr() if need_dw else None, db.data_ptr() if need_dw else None, wp, wn,
                                 _raw_stream(dev, stream))
    if st:
        _check(st, "moe_lora_backward")
    return (dx if need_dx else None), (da if need_dw else None), (db if need_dw else None)


def _stack_out(t, name, dtype, shape, dev):
    import torch
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _stack3d(t, name, dtype, shape, dev)
    if not t.is_contiguous():
        raise MoeError(f"{name}: needs contiguous memory")
    return t
