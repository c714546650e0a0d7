"""Plain 64-bit forms of the dense feed-forward operators and the error
bounds their kernels have to meet.

A bound is what the arithmetic can lose at most, with u = 2^-24 the unit
roundoff of fp32 and e16 that of the 16-bit type (half a step):
  * a sum of n exact products in fp32, in any order: n u sum|a b|;
  * the activation and its derivative in fp32 from a given argument: exp,
    a sum, a reciprocal and a few products. An argument w of the exponential
    carries at most 4 u |w| of rounding, so the sigmoid is good to
    (4 |w| + 8) u relative, which act_u() multiplies out;
  * the result rounded once: e16 |result|, and half a step of the type's
    subnormals.
"""
import math

import torch

U = 2.0 ** -24
E16 = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SUB = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
C = math.sqrt(2.0 / math.pi)


def act(g, name):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(C * (g + 0.044715 * g ** 3)))


def act_d(g, name):
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s + g * s * (1.0 - s)
    t = torch.tanh(C * (g + 0.044715 * g ** 3))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * C * (1.0 + 0.134145 * g * g)


def act_u(g, name):
    """Relative rounding of the sigmoid in units of u (see above)."""
    w = g.abs() if name == "silu" else (2 * C * (g + 0.044715 * g ** 3)).abs()
    # beyond |w| = 90 the sigmoid is 0 or 1 to more than 32 bits
    return 4.0 * w.clamp(max=90.0) + 12.0


def products(x, wg, wu):
    """g, u and the sums of their absolute products."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    return x @ wg.t(), x @ wu.t(), x.abs() @ wg.abs().t(), x.abs() @ wu.abs().t()


def h_bound(g, u, dg, du, name, dt):
    """h = act(g) u from g and u known to dg and du. |act'| <= 1.13 for both
    activations; the second-order part is covered by the factor 1.01."""
    h = act(g, name) * u
    e = 1.01 * (1.13 * dg * (u.abs() + du) + (act(g, name).abs() + 1.13 * dg) * du)
    e = e + h.abs() * act_u(g, name) * U
    return h, e + E16[dt] * (h.abs() + e) + SUB[dt]


def close(got, want, bound, what):
    got = got.double().cpu()
    want, bound = want.cpu(), bound.cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst at "
                           f"{tuple(int(v) for v in bad.nonzero()[0])}: got {got[bad][0].item()!r}, want "
                           f"{want[bad][0].item()!r} +- {bound[bad][0].item():.3e}")


def quant(x):
    """scale (fp32) and codes of the 8-bit rows, from the exact quotient."""
    a = x.float().abs().amax(dim=1).cpu()
    s = torch.where(torch.isfinite(a), a / torch.tensor(127.0), torch.full_like(a, float("nan")))
    z = x.double().cpu()
    ok = (s > 0).unsqueeze(1)
    q = torch.round(z / torch.where(ok, s.double().unsqueeze(1), torch.ones(1, dtype=torch.float64)))
    q = torch.where(ok, q.clamp(-127, 127), torch.zeros_like(z))
    return torch.nan_to_num(q).to(torch.int8), s


def grads(x, wg, wu, gu, dh, name, dt):
    """The gradients and their bounds, from the fp32 g and u that the forward
    call kept (so their rounding is part of the input here)."""
    g, u = gu[:, 0].double(), gu[:, 1].double()
    x, wg, wu, e = x.double(), wg.double(), wu.double(), dh.double()
    dg, du = e * u * act_d(g, name), e * act(g, name)
    # act' = p + g p (1 - p) w': |p (1 - p) g w'| <= 1.2, both terms to act_u
    eg = (e * u).abs() * (1.0 + 1.2) * (act_u(g, name) + 8) * U
    eu = du.abs() * (act_u(g, name) + 2) * U
    I, M = g.shape[1], g.shape[0]
    # rounded to 16 bits, or (up to 32 rows) to a high and a low part: half a
    # step of what half a step leaves
    e16 = E16[dt] if M > 32 else E16[dt] ** 2
    eg = eg + e16 * (dg.abs() + eg) + SUB[dt]
    eu = eu + e16 * (du.abs() + eu) + SUB[dt]
    dx = dg @ wg + du @ wu
    # 2 inter terms (twice: parts), and up to 16 partial sums more
    bx = eg @ wg.abs() + eu @ wu.abs() + (4 * I + 16) * U * ((dg.abs() + eg) @ wg.abs() + (du.abs() + eu) @ wu.abs())
    out = [(dx, bx)]
    for d, b in ((dg, eg), (du, eu)):
        out.append((d.t() @ x, b.t() @ x.abs() + (2 * M + 16) * U * ((d.abs() + b).t() @ x.abs())))
    return [(v, b + E16[dt] * (v.abs() + b) + SUB[dt]) for v, b in out]
