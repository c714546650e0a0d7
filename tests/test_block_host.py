"""Refusals and workspace sizes of the operators around the feed-forward block
through the C ABI, without a GPU: nothing is enqueued on an error, so made-up
pointers of the right alignment serve."""
import ctypes as C
import os

import pytest

qr = pytest.importorskip("quantized_routed_expert_fp32_amd")
B = qr.binding
P = 1 << 20           # never dereferenced
BIG = 1 << 40


def _lib():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return B.lib()


def norm(**kw):
    d = dict(rows=8, hidden=64, dtype=0, x_dtype=0, w_dtype=0, unit_offset=0, eps=1e-6, x=P, ldx=64, residual=None,
             ldresidual=0, w=P)
    d.update(kw)
    return B.NormC(**d)


def lora(**kw):
    d = dict(rows=40000, in_=64, out=32, rank=8, adapters=4, dtype=0, x=P, ldx=64, a=P, lda=64, stride_a=512, b=P, ldb=8,
             stride_b=256, scale=P, ids=P)
    d.update(kw)
    return B.LoraC(**d)


BAD_NORM = [(dict(rows=0), "rows=0", -1), (dict(rows=(1 << 20) + 1), "rows", -1), (dict(hidden=0), "hidden=0", -1),
            (dict(hidden=65537, ldx=65537), "hidden", -1), (dict(dtype=2), "dtype 2", -2), (dict(dtype=16), "dtype 16", -2),
            (dict(x_dtype=1), "x_dtype 1", -2), (dict(w_dtype=1), "w_dtype 1", -2), (dict(x_dtype=16), "without a residual", -2),
            (dict(eps=0.0), "eps", -1), (dict(eps=-1.0), "eps", -1), (dict(eps=float("nan")), "eps", -1),
            (dict(eps=1e-39), "eps", -1), (dict(eps=1.5), "eps", -1), (dict(eps=float("inf")), "eps", -1),
            (dict(unit_offset=2), "unit_offset", -1), (dict(x=None), "NULL x", -1), (dict(w=None), "NULL x/w", -1),
            (dict(ldx=63), "ldx=63", -3), (dict(ldx=(1 << 22) + 1), "ldx", -3)]


@pytest.mark.parametrize("kw,msg,st", BAD_NORM)
def test_norm_refusals(kw, msg, st):
    L = _lib()
    a, n = norm(**kw), C.c_uint64()
    for r in (L.moe_norm_forward(C.byref(a), None, 0, P, 64, None, None),
              L.moe_norm_i8(C.byref(a), None, 0, P, 64, P, None, 0, None),
              L.moe_norm_backward_workspace_size(C.byref(a), C.byref(n)),
              L.moe_norm_backward(C.byref(a), P, P, 64, None, 0, P, 64, P, P, BIG, None)):
        assert r == st
        assert msg in L.moe_last_error().decode()


def test_norm_output_refusals():
    L = _lib()
    err = lambda: L.moe_last_error().decode()
    a, r, n = norm(), norm(residual=P, ldresidual=64), C.c_uint64()
    assert L.moe_norm_forward(None, None, 0, P, 64, None, None) == -1 and "argument block" in err()
    assert L.moe_norm_forward(C.byref(a), None, 0, None, 64, None, None) == -1 and "NULL y" in err()
    assert L.moe_norm_forward(C.byref(a), None, 0, P, 63, None, None) == -3 and "ldy=63" in err()
    assert L.moe_norm_forward(C.byref(a), P, 64, P, 64, None, None) == -1 and "total" in err()
    assert L.moe_norm_forward(C.byref(r), None, 0, P, 64, None, None) == -1 and "total" in err()
    assert L.moe_norm_forward(C.byref(r), P, 60, P, 64, None, None) == -3 and "ldtotal=60" in err()
    b = norm(residual=P, ldresidual=2)
    assert L.moe_norm_forward(C.byref(b), P, 64, P, 64, None, None) == -3 and "ldresidual=2" in err()
    assert L.moe_norm_i8(C.byref(a), None, 0, None, 64, P, None, 0, None) == -1 and "NULL q/scale" in err()
    assert L.moe_norm_i8(C.byref(a), None, 0, P, 64, None, None, 0, None) == -1 and "NULL q/scale" in err()
    assert L.moe_norm_i8(C.byref(a), None, 0, P, 8, P, None, 0, None) == -3 and "ldq=8" in err()
    assert L.moe_norm_i8(C.byref(a), None, 0, P, 64, P, P, 8, None) == -3 and "ldy=8" in err()
    back = lambda a, *v: L.moe_norm_backward(C.byref(a), *v, None)
    assert back(r, P, P, 64, None, 0, P, 64, P, P, BIG) == -1 and "residual" in err()
    assert back(a, None, P, 64, None, 0, P, 64, P, P, BIG) == -1 and "NULL rstd" in err()
    assert back(a, P, None, 64, None, 0, P, 64, P, P, BIG) == -1 and "NULL rstd/dy" in err()
    assert back(a, P, P, 64, None, 0, None, 0, None, P, BIG) == -1 and "no gradient" in err()
    assert back(a, P, P, 64, P, 64, None, 0, P, P, BIG) == -1 and "dtotal without dx" in err()
    assert back(a, P, P, 6, None, 0, P, 64, P, P, BIG) == -3 and "lddy" in err()
    assert back(a, P, P, 64, P, 6, P, 64, P, P, BIG) == -3 and "lddtotal" in err()
    assert back(a, P, P, 64, None, 0, P, 6, P, P, BIG) == -3 and "lddx" in err()
    assert L.moe_norm_backward_workspace_size(C.byref(a), C.byref(n)) == 0 and n.value >= 64 * 4
    assert back(a, P, P, 64, None, 0, P, 64, P, P, n.value - 1) == -4 and str(n.value) in err()
    assert back(a, P, P, 64, None, 0, P, 64, P, None, BIG) == -1 and "NULL ws" in err()
    assert back(a, P, P, 64, None, 0, P, 64, P, P + 16, BIG) == -1 and "aligned" in err()
    assert L.moe_norm_backward_workspace_size(C.byref(a), None) == -1


BALANCE = dict(logits=P, dtype=16, ld=9, ids=P, mask=None, rows=5, experts=8, k=2, losses=P, counts=P, ws=P, n=BIG, s=None)
GRAD = dict(d=P, logits=P, dtype=16, ld=9, mask=None, rows=5, experts=8, k=2, counts=P, out=P, ldd=8, s=None)


@pytest.mark.parametrize("kw,msg,st", [(dict(rows=0), "rows=0", -1), (dict(experts=0), "experts=0", -1),
                                       (dict(experts=1025, ld=1025), "experts=1025", -1), (dict(k=0), "k=0", -1),
                                       (dict(k=9), "k=9", -1), (dict(experts=100, ld=100, k=65), "k=65", -1),
                                       (dict(dtype=2), "dtype 2", -2), (dict(logits=None), "NULL logits", -1),
                                       (dict(ld=7), "ldlogits=7", -3)])
def test_balance_refusals(kw, msg, st):
    L = _lib()
    assert L.moe_balance_forward(*{**BALANCE, **kw}.values()) == st and msg in L.moe_last_error().decode()
    assert L.moe_balance_backward(*{**GRAD, **kw, **({"ldd": 1 << 20} if "experts" in kw else {})}.values()) == st
    assert msg in L.moe_last_error().decode()


def test_balance_output_refusals():
    L = _lib()
    err = lambda: L.moe_last_error().decode()
    for name in ("ids", "losses", "counts"):
        assert L.moe_balance_forward(*{**BALANCE, name: None}.values()) == -1 and "NULL ids/losses/counts" in err()
    for name in ("d", "counts", "out"):
        assert L.moe_balance_backward(*{**GRAD, name: None}.values()) == -1 and "NULL dlosses/counts/dlogits" in err()
    assert L.moe_balance_backward(*{**GRAD, "ldd": 7}.values()) == -3 and "lddlogits=7" in err()
    n = C.c_uint64()
    assert L.moe_balance_workspace_size(5, 8, C.byref(n)) == 0 and n.value
    assert L.moe_balance_forward(*{**BALANCE, "n": n.value - 1}.values()) == -4 and str(n.value) in err()
    assert L.moe_balance_forward(*{**BALANCE, "ws": None}.values()) == -1 and "NULL ws" in err()
    assert L.moe_balance_forward(*{**BALANCE, "ws": P + 8}.values()) == -1 and "aligned" in err()
    assert L.moe_balance_workspace_size(0, 8, C.byref(n)) == -1 and L.moe_balance_workspace_size(8, 2000, C.byref(n)) == -1
    assert L.moe_balance_workspace_size(5, 8, None) == -1


BAD_LORA = [(dict(rows=0), "rows=0", -1), (dict(in_=0), "in=0", -1), (dict(out=65537), "out=65537", -1),
            (dict(rank=0), "rank=0", -1), (dict(rank=257, ldb=257), "rank=257", -1), (dict(adapters=0), "adapters=0", -1),
            (dict(adapters=1025), "adapters=1025", -1), (dict(dtype=16), "dtype 16", -2), (dict(x=None), "NULL", -1),
            (dict(a=None), "NULL", -1), (dict(b=None), "NULL", -1), (dict(scale=None), "NULL", -1),
            (dict(ids=None), "NULL", -1), (dict(ldx=63), "ldx=63", -3), (dict(lda=63), "lda=63", -3),
            (dict(ldb=7), "ldb=7", -3), (dict(stride_a=-1), "stride_a=-1", -3), (dict(stride_b=BIG + 1), "stride_b", -3)]


@pytest.mark.parametrize("kw,msg,st", BAD_LORA)
def test_lora_refusals(kw, msg, st):
    L = _lib()
    a, n = lora(**kw), C.c_uint64()
    for r in (L.moe_lora_workspace_size(C.byref(a), 0, C.byref(n)),
              L.moe_lora_forward(C.byref(a), P, 32, P, 32, None, P, BIG, None),
              L.moe_lora_backward(C.byref(a), P, 32, P, None, 0, P, 64, P, P, P, BIG, None)):
        assert r == st
        assert msg in L.moe_last_error().decode()


def test_lora_output_refusals():
    L = _lib()
    err = lambda: L.moe_last_error().decode()
    a, n = lora(), C.c_uint64()
    fwd = lambda *v: L.moe_lora_forward(C.byref(a), *v, None)
    assert fwd(P, 32, None, 32, None, P, BIG) == -1 and "NULL y" in err()
    assert fwd(P, 31, P, 32, None, P, BIG) == -3 and "ldbase=31" in err()
    assert fwd(None, 0, P, 31, None, P, BIG) == -3 and "ldy=31" in err()
    assert L.moe_lora_workspace_size(C.byref(a), 0, C.byref(n)) == 0 and n.value
    assert fwd(P, 32, P, 32, None, P, n.value - 1) == -4 and str(n.value) in err()
    assert fwd(P, 32, P, 32, None, None, BIG) == -1 and "NULL ws" in err()
    back = lambda *v: L.moe_lora_backward(C.byref(a), *v, None)
    assert back(None, 32, P, None, 0, P, 64, P, P, P, BIG) == -1 and "NULL dy" in err()
    assert back(P, 32, P, None, 0, P, 64, P, None, P, BIG) == -1 and "both" in err()
    assert back(P, 32, P, None, 0, None, 0, None, None, P, BIG) == -1 and "no gradient" in err()
    assert back(P, 32, None, None, 0, P, 64, P, P, P, BIG) == -1 and "NULL t" in err()
    assert back(P, 32, P, P, 64, None, 0, P, P, P, BIG) == -1 and "dx_base without dx" in err()
    assert back(P, 31, P, None, 0, P, 64, P, P, P, BIG) == -3 and "lddy=31" in err()
    assert back(P, 32, P, P, 63, P, 64, P, P, P, BIG) == -3 and "lddx_base=63" in err()
    assert back(P, 32, P, None, 0, P, 63, P, P, P, BIG) == -3 and "lddx=63" in err()
    assert L.moe_lora_workspace_size(C.byref(a), 1, C.byref(n)) == 0
    assert back(P, 32, P, None, 0, P, 64, P, P, P, n.value - 1) == -4 and str(n.value) in err()
    assert back(P, 32, P, None, 0, P, 64, P, P, P + 1, BIG) == -1 and "aligned" in err()
    assert L.moe_lora_workspace_size(C.byref(a), 2, C.byref(n)) == -1 and "kind 2" in err()
    assert L.moe_lora_workspace_size(None, 0, C.byref(n)) == -1 and L.moe_lora_workspace_size(C.byref(a), 0, None) == -1


@pytest.mark.parametrize("rows", [1, 63, 64, 8192, 8193, 1 << 20])
@pytest.mark.parametrize("rank,adapters,dim", [(1, 1, 1), (256, 1024, 64), (64, 16, 65536)])
def test_lora_workspace_covers_its_parts(rows, rank, adapters, dim):
    """At the limits too: no size wraps, and the least that the parts need is there."""
    L = _lib()
    a, n = lora(rows=rows, in_=dim, out=dim, rank=rank, adapters=adapters, ldx=dim, lda=dim, ldb=rank), C.c_uint64()
    assert L.moe_lora_workspace_size(C.byref(a), 1, C.byref(n)) == 0
    rp = -(-rank // 32) * 32
    least = rows * (4 + 4 * rp + 4 + 4 * rank) + (rows // 64 + min(adapters + 1, rows)) * 16
    assert least <= n.value < least + (1 << 45)
    fwd = C.c_uint64()
    assert L.moe_lora_workspace_size(C.byref(a), 0, C.byref(fwd)) == 0 and fwd.value <= n.value
