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


EXPORTS = ["moe_pack_size", "moe_pack_layer_host", "moe_layer_bind", "moe_pack_layer",
           "moe_workspace_size", "moe_route", "moe_experts_decode", "moe_experts_grouped",
           "moe_forward_windows", "moe_forward_windows_noalloc", "moe_route_failures",
           "moe_forward_exact", "moe_glu_workspace_size", "moe_glu_forward", "moe_glu_backward", "moe_glu_i8",
           "moe_quant_rows", "moe_linear_i8_workspace_size", "moe_linear_i8", "moe_status_string", "moe_last_error", "moe_version"]

MOE_WS_DECODE, MOE_WS_GROUPED, MOE_WS_EXACT = 0, 1, 2
MOE_FP32 = 16
MOE_GLU_FORWARD, MOE_GLU_BACKWARD, MOE_GLU_I8 = 0, 1, 2
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
    for f in ("moe_glu_workspace_size", "moe_glu_forward", "moe_glu_backward", "moe_glu_i8", "moe_quant_rows",
              "moe_linear_i8_workspace_size", "moe_linear_i8"):
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
