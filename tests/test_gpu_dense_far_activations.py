"""Activations far below zero, where the sigmoid leaves fp32's normal range
before its product with the gate does: silu(-88) = -5.3e-37 is a normal number.

The bounds are dense_common's, and half a step of fp32's subnormals (2^-150) for
the activation and for its derivative, which are held in fp32.
"""
import pytest
import torch

import dense_common as D
from gpu_common import binding, log
from test_gpu_dense import BF

pytestmark = pytest.mark.gpu


def parts(g, act):
    """The sigmoid, its argument's derivative, the activation and its derivative
    in 64 bits (1 + tanh(w / 2) would cancel where the sigmoid is small)."""
    if act == "silu":
        w, dw = g, torch.ones_like(g)
    else:
        w, dw = 2 * D.C * (g + 0.044715 * g ** 3), 2 * D.C * (1 + 0.134145 * g ** 2)
    p = torch.sigmoid(w)
    return p, dw, g * p, p + g * p * torch.sigmoid(-w) * dw


def gates(act):
    """Gates whose sigmoid's argument runs from -120 to 120."""
    w = torch.linspace(-120, 120, 961, dtype=torch.float64)
    if act == "silu":
        return w.to(BF)
    g = torch.linspace(-12, 12, 961, dtype=torch.float64)
    return g.to(BF)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("rows", [1, 16, 200, 961])
def test_far_gates(rows, act):
    log(f"case far gates {rows} {act}")
    B = binding()
    for first in range(0, 961, rows):
        v = gates(act)[first:first + rows].cuda()
        x = torch.stack([v, torch.ones_like(v)], dim=1).contiguous()           # g = v, u = the column's own
        u = torch.tensor([1.0, -1.0, 0.5, 96.0, 2.0 ** 20, -(2.0 ** 40)], device="cuda", dtype=BF)
        one, zero = torch.ones_like(u), torch.zeros_like(u)
        wg, wu = torch.stack([one, zero], dim=1).contiguous(), torch.stack([zero, u], dim=1).contiguous()
        h, gu = B.glu_forward(x, wg, wu, act=act, save=True)
        g, uu = gu[:, 0].double(), gu[:, 1].double()
        assert torch.equal(g, v.double()[:, None].expand_as(g)) and torch.equal(uu, u.double().expand_as(uu))
        want = parts(g, act)[2] * uu
        e = want.abs() * D.act_u(g, act) * D.U + 2.0 ** -150 * uu.abs()
        D.close(h, want, e + D.E16[BF] * (want.abs() + e) + D.SUB[BF], "h")
        if first > 3 * rows and rows < 16:
            continue
        # the derivative, through dWu's and dWg's single terms: dh = 1, x = (0 but in one row)
        M = v.numel()
        for r in {0, M // 2, M - 1}:
            xr = torch.zeros_like(x)
            xr[r, 0] = 1
            dh = torch.ones(M, 6, device="cuda", dtype=BF)
            _, dwg, dwu = B.glu_backward(dh, xr, wg, wu, gu, act=act, need_dx=False)
            slope, dw, a, d = parts(g[r], act)
            e16 = D.E16[BF] ** 2 if M <= 32 else D.E16[BF]
            for t, want, scale in ((dwg[:, 0], uu[r] * d, uu[r].abs()), (dwu[:, 0], a, torch.ones_like(a))):
                # the sum's rounding is nothing here: one term. The derivative's
                # own: 2.2 p act_u, with p(1 + |g w'|) <= its size where no cancellation is
                size = scale * slope * (1 + g[r].abs() * dw)
                err = size * (D.act_u(g[r], act) + 8) * D.U + 2.0 ** -149 * scale
                err = err + e16 * (want.abs() + err) + D.SUB[BF]
                D.close(t, want, err + D.E16[BF] * (want.abs() + err) + D.SUB[BF], "dw")
