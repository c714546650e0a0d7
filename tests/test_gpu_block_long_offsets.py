"""Operands whose rows lie more than 2^31 elements apart, and calls from two streams at once."""
import pytest
import torch

from gpu_common import binding, log

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LD, ROWS = (1 << 20) + 8, 2100          # 2.2e9 elements between the first row and the last


def far(t):
    """The same values in rows LD elements apart."""
    v = torch.empty(ROWS * LD, device="cuda", dtype=t.dtype).as_strided(t.shape, (LD, 1))
    return v.copy_(t)


def rnd(g, *shape, dt=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def test_norm():
    log("case long norm")
    B, g = binding(), gen(1)
    x, res, w, dy = rnd(g, ROWS, 72, dt=BF), rnd(g, ROWS, 72, dt=BF), rnd(g, 72, dt=BF), rnd(g, ROWS, 72, dt=BF)
    y, total, rstd = B.norm_forward(x, w, residual=res, save=True)
    fy, ft = far(torch.zeros_like(y)), far(res)
    B.norm_forward(far(x), w, residual=ft, total=ft, y=fy)
    assert torch.equal(fy, y) and torch.equal(ft, total)
    q, scale, _, _ = B.norm_i8(x, w, residual=res)
    fq = far(torch.zeros_like(q))
    B.norm_i8(x, w, residual=res, q=fq)
    assert torch.equal(fq, q)
    dx, dw = B.norm_backward(dy, total, w, rstd, dtotal=x)
    B.norm_backward(far(dy), ft, w, rstd, dtotal=x, dx=fy)
    assert torch.equal(fy, dx)


def test_balance():
    log("case long balance")
    B, g = binding(), gen(2)
    l = rnd(g, ROWS, 66, dt=BF)
    ids = l.float().topk(4, dim=1).indices.to(torch.int32)
    d = torch.ones(2, device="cuda")
    losses, counts = B.balance_forward(l, ids)
    dl = B.balance_backward(d, l, counts, 4)
    fl, fd = far(l), far(torch.zeros_like(l))
    got = B.balance_forward(fl, ids)
    assert torch.equal(got[0], losses) and torch.equal(got[1], counts)
    assert torch.equal(B.balance_backward(d, fl, counts, 4, dlogits=fd), dl)


def test_lora():
    log("case long lora")
    B, g = binding(), gen(3)
    x, base, dy, dxb = (rnd(g, ROWS, n, dt=BF) for n in (72, 136, 136, 72))
    n = 1000
    a, b = rnd(g, n, 4, 72, dt=BF), rnd(g, n, 136, 4, dt=BF)
    ids, scale = torch.randint(-1, n, (ROWS,), generator=g, device="cuda").to(torch.int32), torch.ones(n, device="cuda")
    y, t = B.lora_forward(x, a, b, ids, scale, base=base, save=True)
    want = B.lora_backward(dy, x, a, b, ids, scale, t, dx_base=dxb)
    fx, fy = far(x), far(base)
    # adapters 2^22 elements apart
    fa = torch.empty(n << 22, device="cuda", dtype=BF).as_strided(a.shape, (1 << 22, 72, 1)).copy_(a)
    fb = torch.empty(n << 22, device="cuda", dtype=BF).as_strided(b.shape, (1 << 22, 4, 1)).copy_(b)
    B.lora_forward(fx, fa, fb, ids, scale, base=fy, y=fy)
    assert torch.equal(fy, y)
    fdx = far(dxb)
    got = B.lora_backward(far(dy), fx, fa, fb, ids, scale, t, dx_base=fdx, dx=fdx)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    # few rows
    y = B.lora_forward(x[:9], a, b, ids[:9], scale)
    assert torch.equal(B.lora_forward(fx[:9], fa, fb, ids[:9], scale), y)


def test_two_streams_at_once():
    """Each call has a workspace of its own: results as one after the other."""
    log("case two streams")
    B, g = binding(), gen(4)
    R = 3000
    x, w, dy = rnd(g, R, 520, dt=BF), rnd(g, 520, dt=BF), rnd(g, R, 264, dt=BF)
    a, b = rnd(g, 6, 16, 520, dt=BF), rnd(g, 6, 264, 16, dt=BF)
    ids, scale = torch.randint(-1, 6, (R,), generator=g, device="cuda").to(torch.int32), torch.ones(6, device="cuda")
    l = rnd(g, R, 100)
    picks = l.topk(3, dim=1).indices.to(torch.int32)

    def calls(stream):
        y, _, rstd = B.norm_forward(x, w, save=True, stream=stream)
        z, t = B.lora_forward(x, a, b, ids, scale, save=True, stream=stream)
        return (y, z) + B.lora_backward(dy, x, a, b, ids, scale, t, stream=stream) + B.norm_backward(
            x, y, w, rstd, stream=stream) + B.balance_forward(l, picks, stream=stream)

    want = calls(None)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        got += [calls(s) for s in streams]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(p, q) for p, q in zip(r, want))
