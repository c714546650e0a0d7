"""The 8-bit products where the token's and the channel's scale are far from
one: their product alone may leave the range of fp32 where the result does not.
"""
import pytest
import torch

import dense_common as D
from gpu_common import binding, log
from test_gpu_dense import BF, FP, IDS, gen

pytestmark = pytest.mark.gpu

# token scale, channel scale: products far below and above fp32's range, and inside it
SCALES = [(2.0 ** -70 * 1.1, 2.0 ** -70 * 1.3), (2.0 ** -120 * 1.7, 2.0 ** -20 * 1.9), (2.0 ** -20 * 1.7, 2.0 ** -120 * 1.9),
          (2.0 ** -140, 2.0 ** 120 * 1.3), (2.0 ** 120 * 1.9, 2.0 ** -140), (2.0 ** 100, 2.0 ** -100 * 1.7),
          (2.0 ** 90 * 1.5, 2.0 ** 90), (0.013, 0.0021)]


def bound(v, dt):
    # the sum to fp32, the two scales' product, the product with the sum, the
    # result into fp32's subnormals: 4 roundings of u, and half of the smallest fp32
    e = 4 * D.U * v.abs() + 2.0 ** -150
    return e + D.E16[dt] * (v.abs() + e) + D.SUB[dt]


def check_top(y, top):
    """Where |v| (1 + 2^-8) reaches the type's largest value, the result rounded
    by at most half a step is infinite or within 2^-7 of that value: (1 - 2^-8 -
    4 u) / (1 + 2^-8) > 1 - 2^-7."""
    assert (~top | (y.abs() >= torch.finfo(BF).max * (1 - 2.0 ** -7))).all()


def codes(g, r, c):
    return torch.randint(-127, 128, (r, c), generator=g, device="cuda", dtype=torch.int8)


@pytest.mark.parametrize("M,K,N", [(3, 64, 40), (16, 1283, 70), (40, 128, 64), (333, 1283, 777), (700, 8200, 1000),
                                   (1100, 256, 3000)])
def test_linear_i8_scales(M, K, N):
    B = binding()
    g = gen(M + K)
    q, w = codes(g, M, K), codes(g, N, K)
    q[1], w[2] = 0, 0                     # sums of zero: zero, whatever the scales
    acc = q.double() @ w.double().t()
    for a, b in SCALES:
        log(f"case scales {M} {K} {N} {a} {b}")
        s, sw = torch.full((M,), a, device="cuda"), torch.full((N,), b, device="cuda")
        v = acc * s.double()[:, None] * sw.double()
        y = B.linear_i8(q, w, sw, x_scale=s, out_dtype=BF)
        top = v.abs() * (1 + 2.0 ** -8) >= torch.finfo(BF).max
        check_top(y, top)
        assert (y[1] == 0).all() and (y[:, 2] == 0).all()
        D.close(torch.where(top, 0, y.float()), torch.where(top, 0.0, v), bound(v, BF).nan_to_num(posinf=1.0), "y")
        bias = torch.ones(N, device="cuda")
        yb = B.linear_i8(q, w, sw, bias=bias, x_scale=s, out_dtype=BF)
        assert (yb[1] == 1).all() and (yb[:, 2] == 1).all()


@pytest.mark.parametrize("M,H,I", [(2, 64, 40), (16, 1283, 70), (60, 100, 77), (517, 1280, 768), (700, 4100, 1000)])
def test_glu_i8_scales(M, H, I):
    """The gate in range, the up scale far off: h = act(g) u."""
    B = binding()
    g = gen(M + H)
    q, wg, wu = codes(g, M, H), codes(g, I, H), codes(g, I, H)
    ag, au = q.double() @ wg.double().t(), q.double() @ wu.double().t()
    for a, b in SCALES:
        # the gate's scale brings g near one
        sg = float(torch.tensor(2.0 ** -10 / a).clamp(2.0 ** -149, 2.0 ** 127)) / H ** 0.5
        log(f"case scales {M} {H} {I} {a} {b}")
        s = torch.full((M,), a, device="cuda")
        s_g, s_u = torch.full((I,), sg, device="cuda"), torch.full((I,), b, device="cuda")
        gg, uu = ag * s.double()[:, None] * s_g.double(), au * s.double()[:, None] * s_u.double()
        h = B.glu_i8(q, wg, s_g, wu, s_u, x_scale=s, out_dtype=BF)
        eg, eu = 4 * D.U * gg.abs() + 2.0 ** -150, 4 * D.U * uu.abs() + 2.0 ** -150
        want, e = D.h_bound(gg, uu, eg, eu, "silu", BF)
        ok = (uu.abs() < 3e38) & (want.abs() * 1.01 < 3.3e38)      # inside fp32 and the type
        # act(g) u in fp32: below its normal range half of its smallest value
        D.close(torch.where(ok, h.float(), 0), torch.where(ok, want, 0.0), torch.where(ok, e + 2.0 ** -149, 0.0), "h")


@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
def test_small_rows_quantised_in_the_call(dt):
    """Rows of tiny values with weights of large scale, through the quantiser: decode and chunk form."""
    B = binding()
    tiny = 2.0 ** -100 if dt == BF else 2.0 ** -20
    for M in (1, 4, 16, 40, 300):
        g = gen(M)
        x = (torch.randn(M, 512, generator=g, device="cuda") * tiny).to(dt)
        w = codes(g, 100, 512)
        sw = torch.full((100,), 2.0 ** -38 if dt == BF else 2.0 ** 10, device="cuda")
        q, s = D.quant(x)
        v = (q.cuda().double() @ w.double().t()) * s.cuda().double()[:, None] * sw.double()
        D.close(B.linear_i8(x, w, sw), v, bound(v, dt), "y")


@pytest.mark.parametrize("M,K,N", [(5, 64, 40), (40, 128, 64), (333, 1283, 777), (1100, 256, 3000)])
def test_scales_of_every_size_in_one_call(M, K, N):
    """Each row and each channel with a scale of its own, from fp32's smallest values to its largest, zero and NaN among them."""
    log(f"case mixed scales {M} {K} {N}")
    B = binding()
    g = gen(M + K)
    q, w = codes(g, M, K), codes(g, N, K)
    power = lambda n: torch.ldexp(1 + torch.rand(n, generator=g, device="cuda"),
                                  torch.randint(-148, 125, (n,), generator=g, device="cuda"))
    s, sw = power(M), power(N)
    s[0], s[1], sw[3] = 0.0, float("nan"), float("nan")
    v = (q.double() @ w.double().t()) * s.double()[:, None] * sw.double()
    y = B.linear_i8(q, w, sw, x_scale=s, out_dtype=BF)
    assert torch.equal(torch.isnan(y), torch.isnan(v)) and torch.isnan(y[1]).all() and torch.isnan(y[:, 3]).all()
    top = v.abs() * (1 + 2.0 ** -8) >= torch.finfo(BF).max
    check_top(y, top)
    skip = top | torch.isnan(v)
    D.close(torch.where(skip, 0, y.float()), torch.where(skip, 0.0, v), torch.where(skip, 1.0, bound(v, BF)), "y")
    # as the gate or the up product of a gated block
    one = torch.full((N,), 2.0 ** -20, device="cuda")
    for h in (B.glu_i8(q, w, sw, w, one, x_scale=s, out_dtype=BF), B.glu_i8(q, w, one, w, sw, x_scale=s, out_dtype=BF)):
        assert torch.isnan(h[1]).all() and torch.isnan(h[:, 3]).all() and (h[0, 4:] == 0).all()
