"""fp16 gradients of the gated block where dh, and with it dg and du, is far
below the type's normal range: dg and du go into the matrix products scaled by
a power of two a call, so what they lose is relative to the largest of them.

With 2^k the power, k <= 100 the largest that leaves every |dg|, |du| that
fp16 holds below 2^15 (k = 0 at least), the largest is at 2^14 or above, or k =
100. Half a step of the type's subnormals, 2^-25, then counts 2^-25 / 2^k <=
2^-39 max(|dg|, |du|) in dg and du.
"""
import pytest
import torch

import dense_common as D
from gpu_common import binding, log
from test_gpu_dense import block, gen, rnd

pytestmark = pytest.mark.gpu

FP = torch.float16


def grads(x, wg, wu, gu, dh, name):
    """dense_common.grads, with the rounding of dg and du counted as above."""
    g, u = gu[:, 0].double(), gu[:, 1].double()
    x, wg, wu, e = x.double(), wg.double(), wu.double(), dh.double()
    dg, du = e * u * D.act_d(g, name), e * D.act(g, name)
    floor = 2.0 ** -39 * max(dg.abs().max().item(), du.abs().max().item())
    I, M = g.shape[1], g.shape[0]
    e16 = D.E16[FP] if M > 32 else D.E16[FP] ** 2
    eg = (e * u).abs() * 2.2 * (D.act_u(g, name) + 8) * D.U
    eu = du.abs() * (D.act_u(g, name) + 2) * D.U
    eg = eg + e16 * (dg.abs() + eg) + floor
    eu = eu + e16 * (du.abs() + eu) + floor
    bx = eg @ wg.abs() + eu @ wu.abs() + (4 * I + 16) * D.U * ((dg.abs() + eg) @ wg.abs() + (du.abs() + eu) @ wu.abs())
    out = [(dg @ wg + du @ wu, bx)]
    for d, b in ((dg, eg), (du, eu)):
        out.append((d.t() @ x, b.t() @ x.abs() + (2 * M + 16) * D.U * ((d.abs() + b).t() @ x.abs())))
    return [(v, b + D.E16[FP] * (v.abs() + b) + D.SUB[FP]) for v, b in out]


@pytest.mark.parametrize("std", [1e-3, 1e-5, 1e-6, 1e-7])
@pytest.mark.parametrize("M,H,I", [(1, 64, 40), (20, 264, 130), (32, 129, 4096), (100, 72, 512), (512, 2048, 512),
                                   (777, 1283, 769)])
def test_small_dh(M, H, I, std):
    log(f"case small dh {M} {H} {I} {std}")
    B = binding()
    for act in ("silu", "gelu_tanh"):
        x, wg, wu, _ = block(M + H, M, H, I, FP)
        dh = rnd(gen(I), M, I, std=std, dt=FP)
        _, gu = B.glu_forward(x, wg, wu, act=act, save=True)
        got = B.glu_backward(dh, x, wg, wu, gu, act=act)
        for name, t, (want, bound) in zip(("dx", "dw_gate", "dw_up"), got, grads(x, wg, wu, gu, dh, act)):
            D.close(t, want, bound, name)


@pytest.mark.parametrize("j", [7, 13])
@pytest.mark.parametrize("M,H,I", [(17, 96, 200), (200, 136, 520), (2048, 1032, 1500)])
def test_scaled_dh_scales_the_gradients(M, H, I, j):
    """dh 2^-j gives 2^-j times the gradients, bit for bit where those are normal
    numbers of the type (dh in steps of 2^-7 up to 16: exact after the scaling)."""
    log(f"case scaled dh {M} {H} {I} {j}")
    B = binding()
    x, wg, wu, _ = block(M, M, H, I, FP)
    _, gu = B.glu_forward(x, wg, wu, save=True)
    dh = torch.randint(-2 ** 11, 2 ** 11, (M, I), generator=gen(j), device="cuda").to(FP) / 128
    one = B.glu_backward(dh, x, wg, wu, gu)
    small = B.glu_backward(dh * 2.0 ** -j, x, wg, wu, gu)
    for a, b in zip(one, small):
        assert torch.isfinite(a).all() and torch.isfinite(b).all()
        want = a.float() * 2.0 ** -j
        normal = want.abs() >= 2.0 ** -14
        assert normal.any()
        assert torch.equal(b.float()[normal], want[normal])
        # below, two roundings: half a step of the first, half a subnormal step
        assert ((b.float() - want).abs() <= want.abs() * 2.0 ** -11 + 2.0 ** -25).all()


@pytest.mark.parametrize("M", [5, 70])
def test_rows_that_are_not_finite_do_not_count(M):
    """Zero gradients, and rows of NaN, infinity and beyond the type's range: the others as without them."""
    B = binding()
    x, wg, wu, _ = block(M, M, 96, 200, FP)
    _, gu = B.glu_forward(x, wg, wu, save=True)
    for t in B.glu_backward(torch.zeros(M, 200, device="cuda", dtype=FP), x, wg, wu, gu):
        assert (t == 0).all()
    dh = rnd(gen(M), M, 200, std=1e-5, dt=FP)
    dh[2] = 0
    want = B.glu_backward(dh, x, wg, wu, gu, need_dw=False)[0]
    rest = [r for r in range(M) if r != 2]
    for v in (float("nan"), float("inf"), float("-inf")):
        dh[2] = v
        dx = B.glu_backward(dh, x, wg, wu, gu, need_dw=False)[0]
        assert not torch.isfinite(dx[2]).any() and torch.equal(dx[rest], want[rest]), v
    dh[2], gu[2] = 1.0, 1e6
    dx = B.glu_backward(dh, x, wg.abs(), wu.abs(), gu, need_dw=False)[0]
    dh[2] = 0
    want = B.glu_backward(dh, x, wg.abs(), wu.abs(), gu, need_dw=False)[0]
    assert (dx[2] == float("inf")).all() and torch.equal(dx[rest], want[rest])


@pytest.mark.parametrize("M", [9, 300])
def test_replayed_with_other_magnitudes(M):
    """A captured backward pass finds its power of two anew in every replay."""
    B = binding()
    x, wg, wu, _ = block(M, M, 264, 160, FP)
    _, gu = B.glu_forward(x, wg, wu, save=True)
    dh = rnd(gen(1), M, 160, dt=FP)
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        B.glu_backward(dh, x, wg, wu, gu)
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = B.glu_backward(dh, x, wg, wu, gu)
    for i, std in enumerate((1.0, 1e-6, 30.0, 1e-4, 1e-7)):
        dh.copy_(rnd(gen(20 + i), M, 160, std=std, dt=FP))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, B.glu_backward(dh, x, wg, wu, gu)):
            assert torch.equal(a, b), f"replay {i}"
        for name, t, (want, bound) in zip(("dx", "dw_gate", "dw_up"), got, grads(x, wg, wu, gu, dh, "silu")):
            D.close(t, want, bound, name)
