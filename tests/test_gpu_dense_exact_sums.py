"""The dense products on whole numbers, where every sum is exact in fp32 (below
2^24) in any order, so that the results are compared bit for bit: through every
tile, with one K range and with several, in every type (tests/dense_tile_sizes.py).

For the gradients g = 32, where the sigmoid is 1 in fp32 (e^-32 < 2^-25) and so
silu(g) = 32 and silu'(g) = 1 (g p (1 - p) = 4e-13): dg = dh u, du = 32 dh.
"""
import pytest
import torch

import dense_common as D
import dense_tile_sizes as S
from gpu_common import binding, log
from test_gpu_dense import BF, FP, IDS, block, gen

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)


def whole(g, *shape, dt=BF, top=2):
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(dt)


def same(got, want, what):
    assert torch.isfinite(got).all() and got.any(), what
    assert torch.equal(got, want), f"{what}: {int((got != want).sum())} of {want.numel()} differ"


@TYPES
@pytest.mark.parametrize("product,tile,several,M,H,I", S.cases("forward"))
def test_forward(product, tile, several, M, H, I, dt):
    log(f"case exact forward {M} {H} {I} {dt}")
    B = binding()
    g = gen(M + H)
    x, wg, wu = (whole(g, *s, dt=dt) for s in ((M, H), (I, H), (I, H)))
    h, gu = B.glu_forward(x, wg, wu, save=True)
    gg, uu, ag, au = D.products(x, wg, wu)
    assert max(ag.max().item(), au.max().item()) < 2 ** 24
    same(gu[:, 0], gg.float(), "g")
    same(gu[:, 1], uu.float(), "u")
    want, bound = D.h_bound(gg, uu, torch.zeros_like(gg), torch.zeros_like(uu), "silu", dt)
    # what rounds to 65504 or beyond in fp16 (infinity from 65520 on; 32 is a step
    # there) is that or infinite
    top = want.abs() + bound >= 65504 if dt == FP else torch.zeros_like(want, dtype=torch.bool)
    assert (~top | (h.abs() >= 65504 - 32 - 2 * bound)).all() and (h[top].sign() == want[top].sign()).all()
    D.close(torch.where(top, 0, h), torch.where(top, 0.0, want), bound, "h")
    assert torch.equal(B.glu_forward(x, wg, wu), h)


def step(g, M, I, dt):
    """dh and gu of the gradients' cases, and dg and du in 64 bits."""
    dh = whole(g, M, I, dt=dt)
    u = whole(g, M, I).float()
    gu = torch.stack([torch.full_like(u, 32.0), u], dim=1).contiguous()
    e = dh.double()
    return dh, gu, e * u.double(), e * 32


@TYPES
@pytest.mark.parametrize("product,tile,several,M,H,I",
                         S.cases("dx") + [("dx", None, None, M, H, I) for M in (1, 15, 16, 17, 32, 33)
                                          for H, I in ((40, 72), (264, 4100))])
def test_dx(product, tile, several, M, H, I, dt):
    log(f"case exact dx {M} {H} {I} {dt}")
    B = binding()
    g = gen(M + I)
    x, wg, wu = (whole(g, *s, dt=dt) for s in ((M, H), (I, H), (I, H)))
    dh, gu, dg, du = step(g, M, I, dt)
    want = dg @ wg.double() + du @ wu.double()
    assert (dg.abs() @ wg.double().abs() + du.abs() @ wu.double().abs()).max().item() < 2 ** 24
    same(B.glu_backward(dh, x, wg, wu, gu, need_dw=False)[0], want.float().to(dt), "dx")


@TYPES
@pytest.mark.parametrize("product,tile,several,M,H,I",
                         S.cases("dw") + [("dw", None, None, M, H, I) for M in (1, 15, 16, 17, 32, 33, 64, 65)
                                          for H, I in ((40, 72), (520, 300))])
def test_dw(product, tile, several, M, H, I, dt):
    log(f"case exact dw {M} {H} {I} {dt}")
    B = binding()
    g = gen(M + I)
    x, wg, wu = (whole(g, *s, dt=dt) for s in ((M, H), (I, H), (I, H)))
    dh, gu, dg, du = step(g, M, I, dt)
    got = B.glu_backward(dh, x, wg, wu, gu, need_dx=False)[1:]
    for t, d, name in zip(got, (dg, du), ("dw_gate", "dw_up")):
        assert (d.abs().t() @ x.double().abs()).max().item() < 2 ** 24
        same(t, (d.t() @ x.double()).float().to(dt), name)


@pytest.mark.parametrize("M,H,I", [(1 << 20, 8, 8), (1 << 20, 24, 40), (300001, 8, 8), (2596, 1736, 1154), (971, 42, 41),
                                   (3484, 530, 908), (2378, 773, 639), (64, 40, 8), (40, 64, 72), (32, 72, 8), (17, 8, 8)])
@TYPES
def test_dw_counts_every_step_once(M, H, I, dt):
    """One row of each 64 (a K step, or half of one) contributes one, to one
    element of each weight gradient: a step left out, or taken twice, is an
    element that is off by one (32 for the up weight), and the sums are whole
    numbers that both types hold."""
    log(f"case dw steps {M} {H} {I} {dt}")
    B = binding()
    g = gen(M + H)
    n = -(-M // 64)
    row = torch.arange(n, device="cuda") * 64 + torch.randint(0, 64, (n,), generator=g, device="cuda")
    row[-1] = M - 1                                   # the last row of all
    row[0] = 0
    i, c = (torch.randint(0, k, (n,), generator=g, device="cuda") for k in (I, H))
    sign = whole(g, n, top=1).float()
    sign[sign == 0] = 1
    x = whole(g, M, H, dt=dt)
    x[row] = 0
    x[row, c] = 1
    dh = torch.zeros(M, I, device="cuda", dtype=dt)
    dh[row, i] = sign.to(dt)
    gu = torch.ones(M, 2, I, device="cuda")
    gu[:, 0] = 32
    wg, wu = whole(g, I, H, dt=dt), whole(g, I, H, dt=dt)
    want = torch.zeros(I, H, device="cuda", dtype=torch.float64)
    want.index_put_((i, c), sign.double(), accumulate=True)
    assert want.abs().max() <= 256
    for k in {0, n // 2, n - 1}:                      # what the comparison would see without step k
        less = want.clone()
        less[i[k], c[k]] -= sign[k].double()
        assert not torch.equal(less.to(dt), want.to(dt)) and not torch.equal((32 * less).to(dt), (32 * want).to(dt))
    _, dwg, dwu = B.glu_backward(dh, x, wg, wu, gu, need_dx=False)
    same(dwg, want.to(dt), "dw_gate")
    same(dwu, (32 * want).to(dt), "dw_up")


def test_the_longest_dw_on_whole_numbers():
    """2^20 rows of whole numbers: sums up to 2^23 (dg) and 2^22 in steps of 32 (du) by eight workgroups' ranges."""
    B = binding()
    M = 1 << 20
    for H, I in ((8, 8), (264, 40)):
        log(f"case longest dw {H} {I}")
        g = gen(H)
        x, wg, wu = (whole(g, *s) for s in ((M, H), (I, H), (I, H)))
        dh, gu, dg, du = step(g, M, I, BF)
        got = B.glu_backward(dh, x, wg, wu, gu, need_dx=False)[1:]
        for t, d in zip(got, (dg, du)):
            want = d.t() @ x.double()
            same(t, want.float().to(BF), "dw")
            # the last K step missing would show
            assert not torch.equal((want - d[-64:].t() @ x[-64:].double()).float().to(BF), t)


@TYPES
@pytest.mark.parametrize("product,tile,several,M,K,N", S.cases("linear"))
def test_linear_i8(product, tile, several, M, K, N, dt):
    log(f"case exact linear_i8 {M} {K} {N} {dt}")
    B = binding()
    g = gen(M + K)
    q, w = (torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8) for s in ((M, K), (N, K)))
    acc = q.double() @ w.double().t()                # exact
    a = 1.0 if dt == BF else 2.0 ** -10              # in fp16's range, and a power of two
    y = B.linear_i8(q, w, torch.ones(N, device="cuda"), x_scale=torch.full((M,), a, device="cuda"), out_dtype=dt)
    same(y, (acc.float() * a).to(dt), "y")


@TYPES
@pytest.mark.parametrize("product,tile,several,M,H,I", S.cases("glu_i8"))
def test_glu_i8(product, tile, several, M, H, I, dt):
    """Gate sums near 127^2, where silu is the identity in fp32."""
    log(f"case exact glu_i8 {M} {H} {I} {dt}")
    B = binding()
    g = gen(M + H)
    q, wg, wu = (whole(g, *s, dt=torch.int8) for s in ((M, H), (I, H), (I, H)))
    q[:, H // 2] = 127
    wg[:, H // 2] = 127
    gg, uu = q.double() @ wg.double().t(), q.double() @ wu.double().t()
    assert gg.min() > 100
    b = 1.0 if dt == BF else 2.0 ** -10
    one = torch.ones(I, device="cuda")
    h = B.glu_i8(q, wg, one, wu, one * b, x_scale=torch.ones(M, device="cuda"), out_dtype=dt)
    same(h, (gg.float() * (uu.float() * b)).to(dt), "h")


@pytest.mark.parametrize("M", [20, 70])
@TYPES
def test_gradients_against_differences_along_their_signs(M, dt):
    """Along the sign of a gradient the loss sum(dh * h) changes by the sum of its
    absolute values, to which the bounds are small: a central difference in 64
    bits tells the gradient from one that is 15% off (and from zero)."""
    B = binding()
    H, I = 96, 88
    x, wg, wu, dh = block(M, M, H, I, dt)
    for act in ("silu", "gelu_tanh"):
        _, gu = B.glu_forward(x, wg, wu, act=act, save=True)
        got = B.glu_backward(dh, x, wg, wu, gu, act=act)
        bounds = D.grads(x, wg, wu, gu, dh, act, dt)
        args = [t.double() for t in (x, wg, wu)]

        def loss(p):
            return (dh.double() * D.act(p[0] @ p[1].t(), act) * (p[0] @ p[2].t())).sum().item()

        # what the rounding of the kept g and u moves the gradients by (|act'| <= 1.13, |act''| <= 1.2)
        gg, uu, ag, au = D.products(x, wg, wu)
        eg, eu = (H + 16) * D.U * ag, (H + 16) * D.U * au
        e = dh.double().abs()
        ddg, ddu = e * (1.13 * eu + (uu.abs() + eu) * 1.2 * eg), e * 1.13 * eg
        extra = [ddg @ args[1].abs() + ddu @ args[2].abs(), ddg.t() @ args[0].abs(), ddu.t() @ args[0].abs()]
        for k in range(3):
            v = got[k].double().sign()
            eps = 1e-6
            up, dn = (loss([a + s * eps * v if i == k else a for i, a in enumerate(args)]) for s in (1, -1))
            diff, mine = (up - dn) / (2 * eps), got[k].double().abs().sum().item()
            slack = (bounds[k][1] + extra[k]).sum().item() + 1e-6 * abs(diff)
            log(f"sign direction {act} {k}: difference {diff:.6f}, gradient {mine:.6f}, slack {slack:.4f}")
            assert slack < 0.15 * mine and abs(diff - mine) <= slack
