"""Refusals and workspace sizes of the dense feed-forward operators through the
C ABI, without a GPU: nothing is enqueued on an error, so made-up pointers of
the right alignment serve."""
import ctypes as C
import os

import pytest

qr = pytest.importorskip("quantized_routed_expert_fp32_amd")
B = qr.binding
P = 1 << 20           # never dereferenced


def _lib():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return B.lib()


def glu(**kw):
    d = dict(rows=8, hidden=64, inter=32, dtype=0, act=0, w_gate=P, w_up=P, ldw_gate=64, ldw_up=64, s_gate=None,
             s_up=None, x=P, ldx=64, s_x=None)
    d.update(kw)
    return B.GluC(**d)


def linear(**kw):
    d = dict(rows=8, in_=64, out=32, dtype=0, w=P, ldw=64, s_w=P, bias=None, x=P, ldx=64, s_x=None)
    d.update(kw)
    return B.LinearC(**d)


BAD_GLU = [(dict(rows=0), "rows=0", -1), (dict(rows=-1), "rows=-1", -1), (dict(rows=(1 << 20) + 1), "rows", -1),
           (dict(hidden=0), "hidden=0", -1), (dict(hidden=65537, ldx=65537), "hidden", -1), (dict(inter=0), "inter", -1),
           (dict(dtype=2), "dtype 2", -2), (dict(act=5), "act 5", -2), (dict(x=None), "NULL", -1),
           (dict(w_gate=None), "NULL", -1), (dict(w_up=None), "NULL", -1), (dict(ldx=63), "ldx=63", -3),
           (dict(ldw_gate=63), "ldw_gate", -3), (dict(ldw_up=(1 << 22) + 1), "ldw_up", -3),
           (dict(s_gate=P), "scales given", -1), (dict(s_x=P), "scales given", -1)]


@pytest.mark.parametrize("kw,msg,st", BAD_GLU)
def test_glu_refusals(kw, msg, st):
    L = _lib()
    a, n = glu(**kw), C.c_uint64()
    for r in (L.moe_glu_workspace_size(C.byref(a), 0, C.byref(n)), L.moe_glu_forward(C.byref(a), P, 32, None, P, 1 << 30, None),
              L.moe_glu_backward(C.byref(a), P, P, 32, P, 64, P, P, P, 1 << 30, None)):
        assert r == st
        assert msg in L.moe_last_error().decode()


def test_glu_output_refusals():
    L = _lib()
    a, n = glu(rows=40), C.c_uint64()
    err = lambda: L.moe_last_error().decode()
    assert L.moe_glu_forward(C.byref(a), None, 32, None, P, 1 << 30, None) == -1 and "NULL h" in err()
    assert L.moe_glu_forward(C.byref(a), P, 31, None, P, 1 << 30, None) == -3 and "ldh=31" in err()
    assert L.moe_glu_backward(C.byref(a), None, P, 32, P, 64, P, P, P, 1 << 30, None) == -1 and "NULL gu" in err()
    assert L.moe_glu_backward(C.byref(a), P, P, 32, P, 64, P, None, P, 1 << 30, None) == -1 and "both" in err()
    assert L.moe_glu_backward(C.byref(a), P, P, 32, None, 0, None, None, P, 1 << 30, None) == -1 and "no gradient" in err()
    assert L.moe_glu_backward(C.byref(a), P, P, 31, P, 64, P, P, P, 1 << 30, None) == -3 and "lddh" in err()
    assert L.moe_glu_backward(C.byref(a), P, P, 32, P, 63, P, P, P, 1 << 30, None) == -3 and "lddx" in err()
    assert L.moe_glu_workspace_size(C.byref(a), 1, C.byref(n)) == 0 and n.value
    assert L.moe_glu_backward(C.byref(a), P, P, 32, P, 64, P, P, P, n.value - 1, None) == -4
    assert str(n.value) in err()
    assert L.moe_glu_backward(C.byref(a), P, P, 32, P, 64, P, P, None, n.value, None) == -1 and "NULL ws" in err()
    assert L.moe_glu_backward(C.byref(a), P, P, 32, P, 64, P, P, P + 16, n.value, None) == -1 and "aligned" in err()
    assert L.moe_glu_workspace_size(C.byref(a), 3, C.byref(n)) == -1 and "kind 3" in err()
    assert L.moe_glu_workspace_size(None, 0, C.byref(n)) == -1
    assert L.moe_glu_workspace_size(C.byref(a), 0, None) == -1
    assert L.moe_glu_i8(C.byref(a), P, 32, P, 1 << 30, None) == -1 and "s_gate" in err()


def test_workspace_counts_the_copies():
    L = _lib()

    def size(kind=0, **kw):
        n = C.c_uint64()
        a = glu(**kw)
        assert L.moe_glu_workspace_size(C.byref(a), kind, C.byref(n)) == 0, L.moe_last_error()
        return n.value

    big = dict(rows=4096, hidden=512, inter=4096, ldx=512, ldw_gate=512, ldw_up=512)
    assert size(**big) == 0
    x, w = 4096 * 512 * 2, 4096 * 512 * 2
    assert size(**{**big, "x": P + 2}) == x                   # a row start off 16 bytes
    assert size(**{**big, "ldw_up": 515}) == w                # a stride off 16 bytes
    assert size(**{**big, "hidden": 509, "ldx": 512}) == x + 2 * w
    assert size(rows=1) == 0 and size(rows=16, x=P + 2) == 0  # decode rows are read in place
    i8 = dict(s_gate=P, s_up=P)
    assert size(2, **{**big, **i8}) == 4096 * 512 + 4096 * 4
    assert size(2, **{**big, **i8, "s_x": P}) == 0
    d = 4096 * 2 * 4096 * 2
    assert size(1, **big) >= d


@pytest.mark.parametrize("kw,msg,st", [(dict(rows=0), "rows=0", -1), (dict(in_=0), "in=0", -1),
                                       (dict(out=65537), "out=65537", -1), (dict(dtype=16), "dtype 16", -2),
                                       (dict(w=None), "NULL", -1), (dict(s_w=None), "NULL", -1),
                                       (dict(ldx=60), "ldx", -3), (dict(ldw=1), "ldw", -3)])
def test_linear_refusals(kw, msg, st):
    L = _lib()
    a, n = linear(**kw), C.c_uint64()
    for r in (L.moe_linear_i8_workspace_size(C.byref(a), C.byref(n)), L.moe_linear_i8(C.byref(a), P, 32, P, 1 << 30, None)):
        assert r == st
        assert msg in L.moe_last_error().decode()


def test_linear_output_and_quant_refusals():
    L = _lib()
    err = lambda: L.moe_last_error().decode()
    a, n = linear(rows=40), C.c_uint64()
    assert L.moe_linear_i8(C.byref(a), None, 32, P, 1 << 30, None) == -1 and "NULL y" in err()
    assert L.moe_linear_i8(C.byref(a), P, 8, P, 1 << 30, None) == -3 and "ldy=8" in err()
    assert L.moe_linear_i8_workspace_size(C.byref(a), C.byref(n)) == 0 and n.value
    assert L.moe_linear_i8(C.byref(a), P, 32, P, n.value - 1, None) == -4
    q = lambda **k: L.moe_quant_rows(*[{**dict(x=P, dtype=0, rows=4, cols=8, ldx=8, q=P, ldq=8, scale=P, s=None),
                                        **k}[n] for n in ("x", "dtype", "rows", "cols", "ldx", "q", "ldq", "scale", "s")])
    assert q(x=None) == -1 and q(q=None) == -1 and q(scale=None) == -1
    assert q(dtype=2) == -2 and q(rows=0) == -1 and q(cols=0) == -1 and q(ldx=7) == -3 and q(ldq=7) == -3
