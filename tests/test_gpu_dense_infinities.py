"""Gradients of the gated block against weights and rows that are not finite:
infinite where the sum is, NaN where it is, on both sides of the 32 rows up to
which dg and du go into the products as a high and a low part."""
import pytest
import torch

import dense_common as D
from gpu_common import binding, log
from test_gpu_dense import BF, FP, IDS, block

pytestmark = pytest.mark.gpu

INF = float("inf")


def check(got, want, what):
    """Infinities, NaN and finite values in the same places."""
    got, want = got.double(), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    inf = torch.isinf(want)
    assert inf.any() and torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf]), what


@pytest.mark.parametrize("M", [1, 3, 16, 17, 30, 32, 33, 70])
@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
def test_infinite_weights_and_rows(M, dt):
    B = binding()
    for H, I in ((72, 40), (136, 2100)):        # one K range, and several in dx
        log(f"case infinities {M} {H} {I} {dt}")
        x, wg, wu, dh = block(M + H, M, H, I, dt)
        _, gu = B.glu_forward(x, wg, wu, save=True)
        clean = B.glu_backward(dh, x, wg, wu, gu)
        g, u, e = gu[:, 0].double(), gu[:, 1].double(), dh.double()
        dg, du = e * u * D.act_d(g, "silu"), e * D.act(g, "silu")
        # one infinite weight of each matrix in columns of their own, two that meet in a third
        wg2, wu2 = wg.clone(), wu.clone()
        wg2[7, 5], wu2[20, 11] = INF, -INF
        wg2[3, 40], wu2[9, 40] = INF, INF
        dx = B.glu_backward(dh, x, wg2, wu2, gu, need_dw=False)[0]
        want = dg @ wg2.double() + du @ wu2.double()
        check(dx, want, "dx")
        rest = [c for c in range(H) if c not in (5, 11, 40)]
        assert torch.equal(dx[:, rest], clean[0][:, rest])
        # an infinite element of the first and of the last row of x, in columns of their own
        x2 = x.clone()
        x2[0, 6] = INF
        x2[M - 1, 12] = -INF
        x2[0, 50] = x2[M - 1, 50] = INF
        got = B.glu_backward(dh, x2, wg, wu, gu, need_dx=False)[1:]
        rest = [c for c in range(H) if c not in (6, 12, 50)]
        for t, d, c in zip(got, (dg, du), clean[1:]):
            check(t, d.t() @ x2.double(), "dw")
            assert torch.equal(t[:, rest], c[:, rest])
        # a NaN stays in its column
        x2[0, 6] = float("nan")
        got = B.glu_backward(dh, x2, wg, wu, gu, need_dx=False)[1:]
        for t, c in zip(got, clean[1:]):
            assert torch.isnan(t[:, 6]).all() and torch.equal(t[:, rest], c[:, rest])
