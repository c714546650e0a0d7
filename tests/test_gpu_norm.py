"""GPU parity of the norm, its 8-bit form and its gradients against their plain
64-bit forms (tests/block_common.py derives the bounds)."""
import pytest
import torch

import block_common as K
from gpu_common import binding, log

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
IDS = {BF: "bf16", FP: "fp16"}
EPS = 1e-6


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, std=1.0, dt=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)


def check(B, x, w, residual, dt, unit_offset=False, eps=EPS):
    """Forward in both forms and the gradients; returns total."""
    R, H = x.shape
    kw = dict(residual=residual, unit_offset=unit_offset, eps=eps)
    y, total, rstd = B.norm_forward(x, w, save=True, **kw)
    want = K.total_of(x, residual, dt)
    if residual is None:
        assert total is None
    else:
        assert torch.equal(total, want)
    v, bv, rs, brs = K.norm(want, w, eps, dt, unit_offset)
    K.close(rstd, rs, brs, "rstd")
    K.close(y, v, bv, "y")
    assert torch.equal(B.norm_forward(x, w, **kw)[0], y)
    q, scale, t8, y8 = B.norm_i8(x, w, want_y=True, **kw)
    cq, s0 = K.norm_codes(want, w, unit_offset)
    assert torch.equal(q.cpu(), cq)
    s = s0.double() * rs.cpu()
    K.close(scale, s, s0.double() * brs.cpu() + 2 * K.U * s + 2.0 ** -149, "scale")
    assert torch.equal(y8, y) and (t8 is None or torch.equal(t8, want))
    assert torch.equal(B.norm_i8(x, w, **kw)[0], q)
    g = gen(R + H)
    dy = rnd(g, R, H, dt=dt)
    for dtotal in (None, rnd(g, R, H, dt=dt)):
        (dx, bx), (dw, bw) = K.norm_grads(dy, want, w, rstd, dtotal, dt, unit_offset)
        gx, gw = B.norm_backward(dy, want, w, rstd, dtotal=dtotal, unit_offset=unit_offset)
        assert gw.dtype == w.dtype
        K.close(gx, dx, bx, "dx")
        K.close(gw, dw, bw, "dw")
        only, none = B.norm_backward(dy, want, w, rstd, dtotal=dtotal, unit_offset=unit_offset, need_dw=False)
        assert none is None and torch.equal(only, gx)
    none, only = B.norm_backward(dy, want, w, rstd, unit_offset=unit_offset, need_dx=False)
    assert none is None and torch.equal(only, gw)
    return want


# every chunk count of a thread and width of a row's threads, ragged ends, one row to many
SIZES = [(1, 1), (1, 2048), (3, 7), (5, 8), (2, 9), (16, 64), (17, 511), (70, 513), (64, 1283), (33, 2048), (9, 2055),
         (40, 4096), (7, 4097), (3, 8192), (2, 8193), (4, 16385), (2, 32775), (2, 65535), (1, 65536), (1025, 64),
         (1030, 520), (1111, 1283), (1025, 1024), (1027, 2056), (1026, 4095), (1025, 4104), (2100, 2048)]


@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
@pytest.mark.parametrize("R,H", SIZES)
def test_sizes(R, H, dt):
    log(f"case norm {R} {H} {dt}")
    B, g = binding(), gen(R * 3 + H)
    w = (1.0 + rnd(g, H, std=0.3)).to(dt)
    check(B, rnd(g, R, H, dt=dt), w, None, dt)
    check(B, rnd(g, R, H, dt=dt), w, rnd(g, R, H, dt=dt), dt)
    check(B, rnd(g, R, H), w, rnd(g, R, H, dt=dt), dt)


@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
@pytest.mark.parametrize("w32", [False, True])
@pytest.mark.parametrize("unit_offset", [False, True])
@pytest.mark.parametrize("R,H", [(5, 100), (1100, 1000), (3, 5000)])
def test_weights(R, H, dt, w32, unit_offset):
    log(f"case norm weights {R} {H} {dt} {w32} {unit_offset}")
    B, g = binding(), gen(H)
    w = rnd(g, H, std=0.3, dt=F32 if w32 else dt)
    check(B, rnd(g, R, H, dt=dt), w, rnd(g, R, H, dt=dt), dt, unit_offset, eps=0.5)


@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
def test_strides_and_places(dt):
    """Rows at odd addresses and strides, among values that must stay as they are."""
    B, g = binding(), gen(5)
    for R, H in ((5, 77), (1100, 77), (3, 1283), (2, 4100)):
        log(f"case norm strides {R} {H} {dt}")
        view = lambda t: (torch.full((R + 1, H + 5), 7.0, device="cuda", dtype=t)[:R, 3:3 + H])
        x, res, w = view(dt).copy_(rnd(g, R, H)), view(dt).copy_(rnd(g, R, H)), rnd(g, H + 1, dt=dt)[1:]
        x32 = view(F32).copy_(rnd(g, R, H))
        for xx in (x, x32):
            total, y, q = view(dt), view(dt), torch.full((R + 1, H + 5), 7, device="cuda", dtype=torch.int8)
            want = B.norm_forward(xx.contiguous(), w, residual=res.contiguous())
            B.norm_forward(xx, w, residual=res, total=total, y=y)
            assert torch.equal(total, want[1]) and torch.equal(y, want[0])
            y.fill_(1.0)
            B.norm_i8(xx, w, residual=res, total=total, y=y, q=q[:R, 3:3 + H])
            cq = B.norm_i8(xx.contiguous(), w, residual=res.contiguous())[0]
            assert torch.equal(q[:R, 3:3 + H], cq) and torch.equal(y, want[0])
            q[:R, 3:3 + H] = 7
            assert (q == 7).all()
            for t in (total, y):
                whole = t.as_strided((R + 1, H + 5), (H + 5, 1), t.storage_offset() - 3).clone()
                whole[:R, 3:3 + H] = 7.0
                assert (whole == 7.0).all()
        y, total, rstd = B.norm_forward(x, w, residual=res, save=True)
        tv, dy, up, dx = view(dt).copy_(total), view(dt).copy_(rnd(g, R, H)), view(dt).copy_(rnd(g, R, H)), view(dt)
        want = B.norm_backward(dy.contiguous(), total, w, rstd, dtotal=up.contiguous())
        _, dw = B.norm_backward(dy, tv, w, rstd, dtotal=up, dx=dx)
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("R,H", [(1, 2048), (40, 1283), (1100, 777), (1030, 4096), (3, 9000)])
def test_total_in_place(R, H):
    log(f"case norm in place {R} {H}")
    B, g = binding(), gen(H)
    x, res, w = rnd(g, R, H, dt=BF), rnd(g, R, H, dt=BF), rnd(g, H, dt=BF)
    y, total, _ = B.norm_forward(x, w, residual=res)
    for q8 in (False, True):
        for into in (0, 1):
            xx, rr = x.clone(), res.clone()
            t = (xx, rr)[into]
            if q8:
                got = B.norm_i8(xx, w, residual=rr, total=t, want_y=True)[3]
            else:
                got = B.norm_forward(xx, w, residual=rr, total=t)[0]
            assert torch.equal(got, y) and torch.equal(t, total)


@pytest.mark.parametrize("R,H", [(6, 64), (6, 2048), (6, 5000), (1030, 64), (1030, 4096)])
def test_rows_of_extremes(R, H):
    """Zeros, the largest and smallest values of the type, infinities and NaN, each in its own row."""
    log(f"case norm extremes {R} {H}")
    B, g = binding(), gen(3)
    for dt in (BF, FP):
        x, w = rnd(g, R, H, dt=dt), (1.0 + rnd(g, H, std=0.1)).to(dt)
        x[0] = 0
        x[1] = torch.finfo(dt).max * (1 - 2 * (torch.arange(H, device="cuda") % 2)).to(dt)
        x[2] = 2.0 ** -133 if dt == BF else 2.0 ** -24          # the smallest subnormal
        x[3, H // 2] = float("inf")
        x[4, H // 3] = float("nan")
        plain = x.clone()
        plain[3:5] = 1.0
        y, _, rstd = B.norm_forward(x, w, save=True)
        q, scale, _, _ = B.norm_i8(x, w)
        v, bv, rs, brs = K.norm(plain, w, EPS, dt)
        ok = torch.ones(R, dtype=torch.bool, device="cuda")
        ok[3:5] = False
        K.close(rstd[ok], rs[ok], brs[ok], "rstd")
        K.close(y[ok], v[ok], bv[ok], "y")
        assert (y[0] == 0).all() and torch.isfinite(y[ok]).all()
        assert y[3].isnan().sum() == 1 and y[3, H // 2].isnan() and (y[3].nan_to_num() == 0).all() and y[4].isnan().all()
        cq, s0 = K.norm_codes(x, w)
        assert torch.equal(q.cpu(), cq) and scale[0] == 0 and (q[0] == 0).all()
        assert scale[3].isnan() and scale[4].isnan() and (q[3:5] == 0).all()
        # max|v| beyond fp32 (bf16's largest times a weight over 1) is not finite either
        assert bool(scale[1].isnan()) == bool(s0[1].isnan()) and torch.isfinite(scale[2]) and scale[2] > 0


def test_codes_are_those_of_the_quantiser():
    """With weights that are powers of two the codes are quant_rows's of total w, whatever rstd."""
    B, g = binding(), gen(8)
    for R, H in ((1, 2048), (37, 1283), (1200, 512)):
        log(f"case norm codes {R} {H}")
        x, res = rnd(g, R, H, std=3.0, dt=BF), rnd(g, R, H, dt=BF)
        w = torch.exp2(torch.randint(-2, 3, (H,), generator=g, device="cuda").float()).to(BF)
        q, _, total, _ = B.norm_i8(x, w, residual=res)
        assert torch.equal(q, B.quant_rows(total * w)[0])


def test_gradients_against_differences():
    B, g = binding(), gen(4)
    R, H = 3, 40
    x, w, dy = rnd(g, R, H, dt=FP), (1 + rnd(g, H, std=0.2)).to(FP), rnd(g, R, H, dt=FP)
    _, _, rstd = B.norm_forward(x, w, save=True)
    dx, dw = B.norm_backward(dy, x, w, rstd)
    f = lambda xx, ww: (dy.double() * (xx * ww / torch.sqrt((xx * xx).mean(dim=1, keepdim=True) + EPS))).sum()
    h = 1e-6
    xd, wd = x.double(), w.double()
    for t, grad, call in ((xd, dx, lambda v: f(v, wd)), (wd, dw, lambda v: f(xd, v))):
        want = torch.empty_like(t)
        for i in range(t.numel()):
            e = torch.zeros(t.numel(), dtype=torch.float64, device="cuda")
            e[i] = h
            want.view(-1)[i] = (call(t + e.view_as(t)) - call(t - e.view_as(t))) / (2 * h)
        # half a step of the type; the differences' own error (h^2 and 2^-52 / h) is below 1e-8
        K.close(grad, want, K.E16[FP] * want.abs() + 100 * K.U * want.abs().max() + 1e-8, "difference")


def test_streams_and_graphs():
    """On a stream of its own, and captured: replays on new contents of the same memory, with other work between them."""
    B, g = binding(), gen(9)
    R, H = 1100, 1000
    x, res, w, dy = rnd(g, R, H, dt=BF), rnd(g, R, H, dt=BF), rnd(g, H, dt=BF), rnd(g, R, H, dt=BF)

    def call(stream=None):
        y, total, rstd = B.norm_forward(x, w, residual=res, save=True, stream=stream)
        q, scale, _, _ = B.norm_i8(x, w, residual=res, stream=stream)
        dx, dw = B.norm_backward(dy, total, w, rstd, dtotal=res, stream=stream)
        return y, total, q, scale, dx, dw

    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        x.copy_(rnd(g, R, H, dt=BF))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, call())), i
