"""GPU parity of the dense feed-forward operators against their plain 64-bit
forms (tests/dense_common.py derives the bounds)."""
import ctypes as C

import pytest
import torch

import dense_common as D
from gpu_common import binding, log

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
IDS = {BF: "bf16", FP: "fp16"}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, std=1.0, dt=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)


def block(seed, M, H, I, dt):
    g = gen(seed)
    return rnd(g, M, H, dt=dt), rnd(g, I, H, std=H ** -0.5, dt=dt), rnd(g, I, H, std=H ** -0.5, dt=dt), rnd(g, M, I, dt=dt)


def check_forward(x, wg, wu, h, act):
    H = x.shape[1]
    g, u, ag, au = D.products(x, wg, wu)
    want, bound = D.h_bound(g, u, (H + 16) * D.U * ag, (H + 16) * D.U * au, act, x.dtype)
    D.close(h, want, bound, "h")
    return g, u, ag, au


# rows x hidden x inter: one row, decode widths, tile edges, odd sizes, each tile of the products
SIZES = [(1, 64, 8), (1, 2048, 512), (1, 1, 1), (2, 7, 3), (16, 1283, 77), (16, 4096, 130), (17, 64, 64), (17, 8, 1),
         (64, 128, 32), (65, 1280, 96), (33, 131, 67), (200, 200, 200), (257, 1032, 300), (300, 65, 129),
         (1024, 512, 2048), (1100, 264, 1500), (2048, 512, 4100)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
@pytest.mark.parametrize("M,H,I", SIZES)
def test_forward_and_gradients(M, H, I, dt, act):
    log(f"case glu {M} {H} {I} {dt} {act}")
    B = binding()
    x, wg, wu, dh = block(M * 7 + H, M, H, I, dt)
    h = B.glu_forward(x, wg, wu, act=act)
    g, u, ag, au = check_forward(x, wg, wu, h, act)
    h2, gu = B.glu_forward(x, wg, wu, act=act, save=True)
    torch.cuda.synchronize()
    assert torch.equal(h, h2)
    for k, (v, a) in enumerate(((g, ag), (u, au))):
        e = (H + 16) * D.U * a
        D.close(gu[:, k], v, e, "gu")
    got = B.glu_backward(dh, x, wg, wu, gu, act=act)
    for name, t, (want, bound) in zip(("dx", "dw_gate", "dw_up"), got, D.grads(x, wg, wu, gu, dh, act, dt)):
        D.close(t, want, bound, name)
    # one gradient alone: the same bits
    dx, n1, n2 = B.glu_backward(dh, x, wg, wu, gu, act=act, need_dw=False)
    assert n1 is None and n2 is None and torch.equal(dx, got[0])
    n0, dg, du = B.glu_backward(dh, x, wg, wu, gu, act=act, need_dx=False)
    assert n0 is None and torch.equal(dg, got[1]) and torch.equal(du, got[2])


@pytest.mark.parametrize("M,K,N", [(1, 64, 16), (1, 1, 1), (3, 5, 2), (16, 2048, 100), (16, 1283, 33), (17, 16, 5),
                                   (17, 3, 64), (64, 128, 64), (100, 777, 131), (129, 1024, 300), (333, 1283, 777),
                                   (1030, 2048, 2000), (2050, 528, 4100)])
@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
@pytest.mark.parametrize("bias", [False, True])
def test_linear_i8(M, K, N, dt, bias):
    log(f"case linear_i8 {M} {K} {N} {dt} {bias}")
    B = binding()
    g = gen(M + K + N)
    x = rnd(g, M, K, dt=dt)
    w, sw = B.quant_rows(rnd(g, N, K, std=K ** -0.5))
    b = rnd(g, N) if bias else None
    y = B.linear_i8(x, w, sw, bias=b)
    q, s = D.quant(x)
    gq, gs = B.quant_rows(x)
    torch.cuda.synchronize()
    assert torch.equal(gq.cpu(), q) and torch.equal(gs.cpu(), s)
    check_linear(y, q, s, w, sw, b, dt)
    # the same from codes
    assert torch.equal(B.linear_i8(gq, w, sw, bias=b, x_scale=gs, out_dtype=dt), y)


def check_linear(y, q, s, w, sw, b, dt):
    q, s = q.cuda(), s.cpu()
    acc = (q.double() @ w.double().t()).cpu()
    v = acc * s.double().unsqueeze(1) * sw.double().cpu()
    bb = b.double().cpu() if b is not None else torch.zeros(1, dtype=torch.float64)
    # the sum to fp32, two products, the bias added: one rounding each
    e = 4 * D.U * (v.abs() + bb.abs())
    D.close(y, v + bb, e + D.E16[dt] * ((v + bb).abs() + e) + D.SUB[dt], "y")


@pytest.mark.parametrize("M,H,I", [(1, 64, 8), (1, 1, 1), (16, 2048, 130), (15, 1283, 9), (17, 16, 40), (60, 100, 77),
                                   (130, 1280, 256), (517, 1283, 769), (1024, 512, 2048), (2100, 272, 4100)])
@pytest.mark.parametrize("dt,act", [(BF, "silu"), (FP, "gelu_tanh")], ids=["bf16-silu", "fp16-gelu_tanh"])
def test_glu_i8(M, H, I, dt, act):
    log(f"case glu_i8 {M} {H} {I} {dt} {act}")
    B = binding()
    g = gen(M + H + I)
    x = rnd(g, M, H, dt=dt)
    wg, sg = B.quant_rows(rnd(g, I, H, std=H ** -0.5))
    wu, su = B.quant_rows(rnd(g, I, H, std=H ** -0.5))
    h = B.glu_i8(x, wg, sg, wu, su, act=act)
    q, s = D.quant(x)
    qc, sc = q.double().cuda(), s.double().unsqueeze(1).cuda()
    gg, uu = (qc @ w.double().t() * sc * sw.double() for w, sw in ((wg, sg), (wu, su)))
    want, bound = D.h_bound(gg, uu, 4 * D.U * gg.abs(), 4 * D.U * uu.abs(), act, dt)
    D.close(h, want, bound, "h")
    gq, gs = B.quant_rows(x)
    assert torch.equal(B.glu_i8(gq, wg, sg, wu, su, act=act, x_scale=gs, out_dtype=dt), h)


@pytest.mark.parametrize("K", [*range(15, 34), 4095, 4097, 4113])
def test_copied_rows_of_every_length(K):
    """Rows off 16 bytes, of each length modulo 16, among other values: the
    copies hold the row and zeros behind it, whatever stands there."""
    log(f"case copied rows {K}")
    B = binding()
    g = gen(K)
    M, N, pad = 37, 29, -K % 16
    wide = [torch.randint(-127, 128, (r, K + 5), generator=g, device="cuda", dtype=torch.int8) for r in (M, N)]
    s, sw = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    x, w = (t[:, 3:3 + K] for t in wide)
    # the same codes with zeros behind them on 16 bytes: the same exact sums
    xz, wz = (torch.nn.functional.pad(t, (0, pad)) for t in (x, w))
    y = B.linear_i8(x, w, sw, x_scale=s, out_dtype=BF)
    assert torch.equal(y, B.linear_i8(xz, wz, sw, x_scale=s, out_dtype=BF))
    v = rnd(g, M, K + 5, dt=BF)[:, 1:1 + K]              # x quantised in the launch that copies w
    q, qs = B.quant_rows(v)
    assert torch.equal(B.linear_i8(v, w, sw), B.linear_i8(q, w, sw, x_scale=qs, out_dtype=BF))
    for dt in (BF, FP):
        f = [torch.full((r, K + 3), float("nan"), device="cuda", dtype=dt) for r in (M, N, N)]
        x, wg, wu = (t[:, 1:1 + K] for t in f)
        for t, a in zip((x, wg, wu), block(K, M, K, N, dt)):
            t.copy_(a)
        h, gu = B.glu_forward(x, wg, wu, save=True)
        check_forward(x, wg, wu, h, "silu")
        dh = rnd(g, M, N, dt=dt)
        got = B.glu_backward(dh, x, wg, wu, gu)
        for name, t, (want, bound) in zip(("dx", "dw_gate", "dw_up"), got, D.grads(x, wg, wu, gu, dh, "silu", dt)):
            D.close(t, want, bound, name)


# sizes that take each tile of the products with one K range and with several:
# 256 x 256, 128 x 128 (both step widths) and 64 x 64, in the forward products
# and in each gradient, ragged in every dimension
TILES = [(4000, 1300, 2000), (700, 2056, 2000), (2000, 4100, 300), (520, 4104, 2060), (40, 8200, 520), (2048, 512, 4100),
         (700, 4100, 1000), (100, 200, 9000), (2500, 3000, 40), (9000, 520, 520)]


@pytest.mark.parametrize("M,H,I", TILES)
def test_every_tile(M, H, I):
    log(f"case tiles {M} {H} {I}")
    B = binding()
    dt, act = BF, "silu"
    x, wg, wu, dh = block(M + H + I, M, H, I, dt)
    h, gu = B.glu_forward(x, wg, wu, act=act, save=True)
    check_forward(x, wg, wu, h, act)
    got = B.glu_backward(dh, x, wg, wu, gu, act=act)
    for name, t, (want, bound) in zip(("dx", "dw_gate", "dw_up"), got, D.grads(x, wg, wu, gu, dh, act, dt)):
        D.close(t, want, bound, name)
    again = B.glu_backward(dh, x, wg, wu, gu, act=act)
    assert torch.equal(B.glu_forward(x, wg, wu, act=act), h)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    (q, s), (w, sw), (v, sv) = B.quant_rows(x), B.quant_rows(wg), B.quant_rows(wu)
    check_linear(B.linear_i8(x, w, sw), q, s, w, sw, None, dt)
    qc, sc = q.double(), s.double().unsqueeze(1)
    gg, uu = (qc @ m.double().t() * sc * sm.double() for m, sm in ((w, sw), (v, sv)))
    want, bound = D.h_bound(gg, uu, 4 * D.U * gg.abs(), 4 * D.U * uu.abs(), act, dt)
    D.close(B.glu_i8(x, w, sw, v, sv, act=act), want, bound, "h")


@pytest.mark.parametrize("M", [1, 15, 16, 17, 31, 32, 33])
@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
def test_gradients_of_few_rows(M, dt):
    """On both sides of the 32 rows up to which dg and du go as high and low
    parts (the bounds of the gradients count them), with one K range and several."""
    B = binding()
    for H, I in ((72, 40), (264, 4096), (1001, 129)):
        log(f"case few rows {M} {H} {I} {dt}")
        x, wg, wu, dh = block(M * H, M, H, I, dt)
        _, gu = B.glu_forward(x, wg, wu, save=True)
        got = B.glu_backward(dh, x, wg, wu, gu)
        for name, t, (want, bound) in zip(("dx", "dw_gate", "dw_up"), got, D.grads(x, wg, wu, gu, dh, "silu", dt)):
            D.close(t, want, bound, name)
    # a gradient beyond the type's range: infinite, not NaN, and in its own row
    if dt == FP:
        x, wg, wu, dh = block(1, M, 64, 32, dt)
        gu = B.glu_forward(x, wg, wu, save=True)[1]
        gu[0] = 1e6          # act' = 1, so dg = 1e6: infinite in fp16, and so is act(g)
        dx = B.glu_backward(torch.ones_like(dh), x, torch.ones_like(wg), torch.ones_like(wu), gu, need_dw=False)[0]
        assert (dx[0] == float("inf")).all() and torch.isfinite(dx[1:]).all()


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 15, 16])
def test_decode_rows_of_8_bit_weights(M):
    """Every row count of the decode form, on both sides of the size up to which
    it quantises x itself; a row's result does not depend on the others'."""
    B = binding()
    g = gen(M)
    for K in (16, 250, 16384 // M, 16384 // M + 1, 5000):
        log(f"case decode {M} {K}")
        x = rnd(g, M, K, dt=BF)
        w, sw = B.quant_rows(rnd(g, 70, K, std=K ** -0.5))
        y = B.linear_i8(x, w, sw)
        q, s = D.quant(x)
        check_linear(y, q, s, w, sw, None, BF)
        for r in (0, M - 1):
            assert torch.equal(B.linear_i8(x[r:r + 1], w, sw)[0], y[r])


def test_longest_contraction():
    """in = 65536, the most that int32 sums of 127^2 hold, decode and chunk form."""
    B = binding()
    K = 65536
    w = torch.full((5, K), 127, dtype=torch.int8, device="cuda")
    w[1] = -127
    w[2, ::2] = -127
    sw = torch.ones(5, device="cuda")
    for M in (2, 40):
        x = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
        y = B.linear_i8(x, w, sw, x_scale=torch.full((M,), 2.0 ** -30, device="cuda"))
        top = torch.tensor(127.0 * 127 * K * 2.0 ** -30).bfloat16()       # 127^2 K has 14 significant bits: exact in fp32
        want = torch.stack([top, -top, 0 * top, top, top]).cuda()
        assert torch.equal(y, want.expand(M, 5))
        h = B.glu_i8(x, w[:1], sw[:1] * 0 + 1e-9, w[2:3], sw[:1], x_scale=torch.ones(M, device="cuda"))
        assert (h == 0).all()


def test_most_rows():
    """2^20 rows through every kernel with a workgroup a row."""
    B = binding()
    M, H, I = 1 << 20, 8, 8
    x, wg, wu, dh = block(3, M, H, I, BF)
    h, gu = B.glu_forward(x, wg, wu, save=True)
    check_forward(x, wg, wu, h, "silu")
    got = B.glu_backward(dh, x, wg, wu, gu)
    for name, t, (want, bound) in zip(("dx", "dw_gate", "dw_up"), got, D.grads(x, wg, wu, gu, dh, "silu", BF)):
        D.close(t, want, bound, name)
    w, sw = B.quant_rows(wg)
    y = B.linear_i8(x, w, sw)
    check_linear(y, *D.quant(x), w, sw, None, BF)
    assert torch.equal(y[-7:], B.linear_i8(x[-7:], w, sw))


def test_calls_at_once():
    """Calls on two streams at once, each with its own workspace, and two graphs replayed at once."""
    B = binding()
    sets = [block(60 + i, 300 + 50 * i, 520, 264, BF) for i in range(2)]

    def step(s):
        x, wg, wu, dh = s
        h, gu = B.glu_forward(x, wg, wu, save=True)
        w, sw = B.quant_rows(wu)
        return (h, *B.glu_backward(dh, x, wg, wu, gu), B.linear_i8(x, w, sw))

    want = [step(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    for st, s in zip(streams, sets):
        with torch.cuda.stream(st):
            step(s)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(s))
        graphs.append(g)
    for _ in range(3):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(step(s))
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for w, a, b in zip(want, got, outs):
            for t, u, v in zip(w, a, b):
                assert torch.equal(t, u) and torch.equal(t, v)


def test_quant_rows_borders_and_extremes():
    """Ties, rows of zeros, the smallest and largest values, infinities and NaN."""
    B = binding()
    half = torch.arange(-127, 127, device="cuda").float() + 0.5
    rows = [torch.cat([half, torch.tensor([127.0, -127.0], device="cuda")]),      # scale 1: exact ties
            torch.zeros(256, device="cuda"),
            torch.linspace(-1, 1, 256, device="cuda"),
            torch.full((256,), 3.3e38, device="cuda"),
            torch.linspace(0, 1e-38, 256, device="cuda"),
            torch.linspace(0, 1e-43, 256, device="cuda"),
            torch.full((256,), 1e-45, device="cuda")]
    rows += [r * s for s in (1 / 3, 7.7e-6, 1.9e12) for r in rows[:1]]
    x = torch.stack(rows)
    for dt in (torch.float32, BF, FP):
        xv = x.to(dt)
        keep = torch.isfinite(xv).all(dim=1)
        xv = xv[keep].contiguous()
        q, s = B.quant_rows(xv)
        wq, wsc = D.quant(xv)
        assert torch.equal(q.cpu(), wq), dt
        assert torch.equal(s.cpu(), wsc), dt
    for bad in (float("inf"), -float("inf"), float("nan")):
        xv = torch.randn(3, 100, device="cuda")
        xv[1, 57] = bad
        q, s = B.quant_rows(xv)
        assert torch.isnan(s[1]) and not q[1].any() and torch.isfinite(s[[0, 2]]).all()
        w, sw = B.quant_rows(torch.randn(40, 100, device="cuda"))
        y = B.linear_i8(xv.to(BF), w, sw)
        assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2]]).all()


@pytest.mark.parametrize("M", [5, 70, 600])
def test_strided_misaligned_operands(M):
    """Rows inside larger tensors: any row stride and start; what lies between is
    neither read (NaN there) nor written."""
    B = binding()
    dt, H, I = BF, 256, 136
    g = gen(M)

    def inside(rows, cols, left, right, kind=dt):
        if kind == torch.int8:
            t = torch.full((rows + 2, left + cols + right), 99, dtype=kind, device="cuda")
            v = torch.randint(-127, 128, (rows, cols), generator=g, device="cuda").to(kind)
        else:
            t = torch.full((rows + 2, left + cols + right), float("nan"), dtype=kind, device="cuda")
            v = rnd(g, rows, cols, std=0.2, dt=kind)
        t[1:1 + rows, left:left + cols] = v
        return t, t[1:1 + rows, left:left + cols]

    for left, right in ((8, 8), (1, 0), (0, 3), (3, 5)):
        log(f"case strided {M} {left} {right}")
        _, x = inside(M, H, left, right)
        _, wg = inside(I, H, right, left)
        _, wu = inside(I, H, left, right + 16)
        _, dh = inside(M, I, left, right)
        hb, hv = inside(M, I, left, right)
        xb, dxv = inside(M, H, left, right)
        hb.fill_(7.0)
        xb.fill_(7.0)
        h, gu = B.glu_forward(x, wg, wu, save=True, h=hv)
        dx, dg, du = B.glu_backward(dh, x, wg, wu, gu, dx=dxv)
        c = [t.contiguous() for t in (x, wg, wu, dh)]
        h2, gu2 = B.glu_forward(*c[:3], save=True)
        r2 = B.glu_backward(c[3], *c[:3], gu2)
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and torch.equal(gu, gu2)
        for a, b in zip((dx, dg, du), r2):
            assert torch.equal(a, b)
        for buf, n in ((hb, I), (xb, H)):
            m = torch.ones_like(buf, dtype=torch.bool)
            m[1:1 + M, left:left + n] = False
            assert (buf[m] == 7.0).all()
        _, w = inside(I, H, left, right, torch.int8)
        _, q = inside(M, H, right, left, torch.int8)
        sw, sx = torch.rand(I, generator=g, device="cuda"), torch.rand(M, generator=g, device="cuda")
        assert torch.equal(B.linear_i8(q, w, sw, x_scale=sx),
                           B.linear_i8(q.contiguous(), w.contiguous(), sw, x_scale=sx))
        assert torch.equal(B.linear_i8(x, w, sw), B.linear_i8(x.contiguous(), w.contiguous(), sw))


@pytest.mark.parametrize("M", [3, 40, 500])
def test_nan_and_infinity_stay_in_their_rows(M):
    B = binding()
    x, wg, wu, dh = block(M, M, 192, 72, BF)
    clean, gu0 = B.glu_forward(x, wg, wu, save=True)
    x2 = x.clone()
    x2[1, 5] = float("nan")
    x2[2, 100] = float("inf")
    h, gu = B.glu_forward(x2, wg, wu, save=True)
    keep = [r for r in range(M) if r not in (1, 2)]
    assert torch.isnan(h[1]).all() and not torch.isfinite(h[2]).all()
    assert torch.equal(h[keep], clean[keep])
    d0 = B.glu_backward(dh, x, wg, wu, gu0)[0]
    e = dh.clone()
    e[1] = float("nan")
    dx, dg, _ = B.glu_backward(e, x, wg, wu, gu0)
    rest = [r for r in range(M) if r != 1]
    assert torch.isnan(dx[1]).all() and torch.equal(dx[rest], d0[rest]) and torch.isnan(dg).all()
    # a weight row that is not finite spoils its own output column only
    wn = wg.clone()
    wn[7, 3] = float("nan")
    h = B.glu_forward(x, wn, wu)
    cols = [c for c in range(72) if c != 7]
    assert torch.isnan(h[:, 7]).all() and torch.equal(h[:, cols], clean[:, cols])


def test_large_activations():
    """Pre-activations far from zero: the sigmoid saturates without NaN, forward and backward."""
    B = binding()
    for dt, big in ((BF, 1e30), (FP, 200.0)):
        for act in ("silu", "gelu_tanh"):
            x = torch.tensor([[1.0], [-1.0], [1e-3]], device="cuda").repeat(7, 1).to(dt)
            wg = torch.full((40, 1), big, device="cuda").to(dt)
            wu = torch.ones(40, 1, device="cuda").to(dt)
            h, gu = B.glu_forward(x, wg, wu, act=act, save=True)
            dx, dg, du = B.glu_backward(torch.ones_like(h), x, wg, wu, gu, act=act)
            assert torch.equal(h[0], (x[0] * wg[:, 0]) * x[0]) and (h[1] == 0).all()
            assert not torch.isnan(dg).any() and not torch.isnan(du).any() and not torch.isnan(dx).any()


def test_streams_and_repeated_calls():
    """On another stream than the current one, and with one workspace for calls in turn."""
    B = binding()
    x, wg, wu, dh = block(11, 100, 520, 200, BF)
    h0, gu0 = B.glu_forward(x, wg, wu, save=True)
    g0 = B.glu_backward(dh, x, wg, wu, gu0)
    w, sw = B.quant_rows(wg)
    y0 = B.linear_i8(x, w, sw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    n = max(B.glu_workspace_size(x, wg, wu, k) for k in (B.MOE_GLU_FORWARD, B.MOE_GLU_BACKWARD)) + (1 << 20)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        h, gu = B.glu_forward(x, wg, wu, save=True, ws=ws, stream=s)
        g = B.glu_backward(dh, x, wg, wu, gu, ws=ws, stream=s)
        y = B.linear_i8(x, w, sw, ws=ws, stream=s)
        s.synchronize()
        assert torch.equal(h, h0) and torch.equal(y, y0)
        for a, b in zip(g, g0):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [4, 90])
def test_captured_and_replayed(M):
    """A captured training step and 8-bit chain replay with new inputs, eager work between the replays."""
    B = binding()
    H, I = 384, 160
    x, wg, wu, dh = block(5, M, H, I, BF)
    w8, s8 = B.quant_rows(rnd(gen(3), H, I))

    def step():
        h, gu = B.glu_forward(x, wg, wu, save=True)
        return (h, *B.glu_backward(dh, x, wg, wu, gu), B.linear_i8(h, w8, s8))

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        nx, _, _, ne = block(50 + i, M, H, I, BF)
        x.copy_(nx)
        dh.copy_(ne)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), f"replay {i}"


@pytest.mark.parametrize("M", [9, 150])
def test_feed_forward_of_8_bit_weights(M):
    """The operators in a row, as an 8-bit feed-forward block runs: the rows to
    codes, the gated block, its output through the down projection."""
    B = binding()
    H, I, dt = 512, 384, BF
    g = gen(M)
    x = rnd(g, M, H, dt=dt)
    gate, up = (B.quant_rows(rnd(g, I, H, std=H ** -0.5)) for _ in range(2))
    down = B.quant_rows(rnd(g, H, I, std=I ** -0.5))
    q, s = B.quant_rows(x)
    h = B.glu_i8(q, *gate, *up, x_scale=s, out_dtype=dt)
    y = B.linear_i8(h, *down)
    assert torch.equal(h, B.glu_i8(x, *gate, *up))
    hq, hs = D.quant(h)
    check_linear(y, hq, hs, *down, None, dt)
    # against the block on the unquantised values the codes stand for
    xv = q.double() * s.double().unsqueeze(1)
    dq = lambda p: p[0].double() * p[1].double().unsqueeze(1)
    hv = D.act(xv @ dq(gate).t(), "silu") * (xv @ dq(up).t())
    # h to 16 bits and to 8: half a step of its row's scale, and the bf16 half step
    eh = hs.double().cuda().unsqueeze(1) * 0.5 + hv.abs() * 2.0 ** -8 * 1.01 + hs.double().cuda().unsqueeze(1) * 2.0 ** -7
    want = hv @ dq(down).t()
    e = eh @ dq(down).abs().t()
    D.close(y, want, e * 1.01 + want.abs() * 2.0 ** -8, "y")


def test_gradients_against_differences():
    """The kernels' gradients along a direction against a central difference
    of the 64-bit loss sum(dh * h) (its own error: eps^2 times a third derivative)."""
    B = binding()
    M, H, I, dt = 70, 96, 88, FP
    x, wg, wu, dh = block(2, M, H, I, dt)
    g = gen(9)
    for act in ("silu", "gelu_tanh"):
        h, gu = B.glu_forward(x, wg, wu, act=act, save=True)
        got = B.glu_backward(dh, x, wg, wu, gu, act=act)
        bounds = D.grads(x, wg, wu, gu, dh, act, dt)
        args = [t.double() for t in (x, wg, wu)]

        def loss(p):
            a, b, c = p
            return (dh.double() * D.act(a @ b.t(), act) * (a @ c.t())).sum().item()

        # the kernel starts from the fp32 sums g and u: what their rounding moves
        # the gradients by, bounded through |act'| <= 1.13, |act''| <= 1.2
        gg, uu, ag, au = D.products(x, wg, wu)
        eg, eu = (H + 16) * D.U * ag, (H + 16) * D.U * au
        e = dh.double().abs()
        ddg, ddu = e * (1.13 * eu + (uu.abs() + eu) * 1.2 * eg), e * 1.13 * eg
        extra = [ddg @ args[1].abs() + ddu @ args[2].abs(), ddg.t() @ args[0].abs(), ddu.t() @ args[0].abs()]
        for k in range(3):
            v = rnd(g, *args[k].shape).double()
            eps = 1e-5
            up = loss([a + eps * v if i == k else a for i, a in enumerate(args)])
            dn = loss([a - eps * v if i == k else a for i, a in enumerate(args)])
            diff = (up - dn) / (2 * eps)
            mine = (got[k].double() * v).sum().item()
            slack = ((bounds[k][1] + extra[k]) * v.abs()).sum().item() + 1e-6 * abs(diff) + 1e-6
            log(f"direction {act} {k}: difference {diff:.6f}, gradient {mine:.6f}, slack {slack:.4f}")
            assert abs(diff - mine) <= slack


def test_refusals_enqueue_nothing():
    B = binding()
    x, wg, wu, dh = block(1, 4, 64, 32, BF)
    h, gu = B.glu_forward(x, wg, wu, save=True)
    w, sw = B.quant_rows(wg)
    bad = [
        (lambda: B.glu_forward(x.float(), wg, wu), "x: dtype"),
        (lambda: B.glu_forward(x, wg.half(), wu), "w_gate: dtype"),
        (lambda: B.glu_forward(x, wg, wu[:31]), "w_up: shape"),
        (lambda: B.glu_forward(x[:, :60], wg, wu), "w_gate has 64 columns"),
        (lambda: B.glu_forward(x.t(), wg, wu), "contiguous"),
        (lambda: B.glu_forward(x[0], wg, wu), "1-D"),
        (lambda: B.glu_forward(x, wg, wu, act="relu"), "act"),
        (lambda: B.glu_forward(x, wg.cpu(), wu), "needs device memory"),
        (lambda: B.glu_forward(x[:0], wg, wu), "rows=0"),
        (lambda: B.glu_forward(x, wg, wu, h=h.float()), "h: dtype"),
        (lambda: B.glu_backward(dh, x, wg, wu, gu[:3]), "gu"),
        (lambda: B.glu_backward(dh[:3], x, wg, wu, gu), "dh: shape"),
        (lambda: B.glu_backward(dh, x, wg, wu, gu, need_dx=False, need_dw=False), "neither"),
        (lambda: B.glu_backward(dh, x, wg, wu, gu, ws=torch.empty(256, dtype=torch.uint8, device="cuda")),
         "MOE_ENOSPACE"),
        (lambda: B.glu_i8(x, w, sw[:5], w, sw), "s_gate"),
        (lambda: B.glu_i8(x, wg, sw, wu, sw), "w_gate: dtype"),
        (lambda: B.linear_i8(x, w, sw.double()), "s_w"),
        (lambda: B.linear_i8(x, w, sw, bias=sw[:3]), "bias"),
        (lambda: B.linear_i8(w, w, sw), "x: dtype"),
        (lambda: B.linear_i8(x, w, sw, out_dtype=FP), "out_dtype"),
        (lambda: B.quant_rows(w), "x: dtype"),
    ]
    for f, what in bad:
        with pytest.raises(B.MoeError, match=what):
            f()
