"""Plain 64-bit forms of the operators around the feed-forward block and the
error bounds their kernels have to meet, from the same units as
tests/dense_common.py: u = 2^-24, e16 half a step of the 16-bit type, a sum of n
terms in fp32 in any order n u sum|terms| (n + 1 where the terms are products
that are rounded themselves). An fp32 product, quotient or root adds u of its value.
"""
import math

import torch

import dense_common as D
from dense_common import E16, SUB, U, quant  # noqa: F401


def close(got, want, bound, what):
    """dense_common's, where a value of 65520 and more (half a step above fp16's largest) is its infinity."""
    if got.dtype == torch.float16:
        far = want.abs() + bound >= 65520
        inf = torch.copysign(torch.full_like(want, math.inf), want)
        sure = want.abs() - bound >= 65520
        assert torch.equal(got[sure].double(), inf[sure]), what
        either = far & (got.double() == inf)
        got, want = torch.where(either, 0, got), torch.where(either, 0, want)
    D.close(got, want, bound, what)


def rounded(v, e, dt):
    """A bound e on a value, after its rounding to dt."""
    if dt == torch.float32:
        return e + U * (v.abs() + e) + 2.0 ** -149
    return e + E16[dt] * (v.abs() + e) + SUB[dt]


# ------------------------------------------------------------------- norm
def total_of(x, residual, dt):
    return x if residual is None else (x.float() + residual.float()).to(dt)


def weight_of(w, unit_offset):
    """The weights as the kernel has them: 1 + w is rounded to fp32."""
    return (1.0 + w.float() if unit_offset else w.float()).double()


def norm(total, w, eps, dt, unit_offset=False):
    """(y, its bound, rstd, its bound). The mean is off by H + 1 roundings (its division one more),
    half of that after the root, which adds two of its own."""
    s, H = total.double(), total.shape[1]
    rs = 1.0 / torch.sqrt((s * s).mean(dim=1, keepdim=True) + float(torch.tensor(eps)))
    rel = ((H + 3) / 2 + 2) * U
    y = s * rs * weight_of(w, unit_offset)
    return y, rounded(y, (rel + 2 * U) * y.abs(), dt), rs.squeeze(1), rel * rs.squeeze(1) + 2.0 ** -149


def norm_codes(total, w, unit_offset=False):
    """Codes and s0 of v = fp32(total w)."""
    w = 1.0 + w.float() if unit_offset else w.float()
    return quant(total.float() * w)


def norm_grads(dy, total, w, rstd, dtotal, dt, unit_offset=False):
    """((dx, bound), (dw, bound)) for the fp32 rstd that the forward call kept. n = total
    rstd is rounded once; a term of the dot product is three products."""
    e, s, rs = dy.double(), total.double(), rstd.double().unsqueeze(1)
    R, H = s.shape
    wv = weight_of(w, unit_offset)
    n = s * rs
    terms = e * wv * n
    dot = terms.sum(dim=1, keepdim=True) / H
    ddot = (H + 4) * U * terms.abs().sum(dim=1, keepdim=True) / H
    up = torch.zeros_like(e) if dtotal is None else dtotal.double()
    dx = rs * (e * wv - n * dot) + up
    sizes = rs * ((e * wv).abs() + n.abs() * (dot.abs() + ddot))
    bx = rs * n.abs() * ddot + 6 * U * sizes + U * (sizes + up.abs())
    dw = (e * n).sum(dim=0)
    bw = (R + 3) * U * (e * n).abs().sum(dim=0)
    return (dx, rounded(dx, bx, dt)), (dw, rounded(dw, bw, w.dtype))


# ---------------------------------------------------------------- balance
def balance(logits, ids, mask, dlosses):
    """(losses, bound), counts, (dlogits, bound). The exponential's argument is rounded once (so
    its value is off by u |l - top|, and 2 u of its own); a value below e^-105 is zero in fp32."""
    R, E = logits.shape
    k = ids.shape[1]
    keep = torch.ones(R, dtype=torch.bool, device=logits.device) if mask is None else mask
    l, i = logits[keep].double(), ids[keep].long()
    n = l.shape[0]
    counts = torch.zeros(E + 1, dtype=torch.int64, device=logits.device)
    i = i[(i >= 0) & (i < E)]
    counts[:E] = (i.reshape(-1, 1) == torch.arange(E, device=i.device)).sum(dim=0)
    counts[E] = n
    d = torch.zeros(R, E, dtype=torch.float64, device=logits.device)
    bd = torch.zeros_like(d)
    if n == 0:
        z = torch.zeros(2, dtype=torch.float64, device=logits.device)
        return (z, z), counts.int(), (d, bd)
    top = l.amax(dim=1, keepdim=True)
    far = (top - l).clamp(max=105.0)
    lse = torch.logsumexp(l, dim=1, keepdim=True)
    p = torch.exp(l - lse)
    # e^(l - top): far + 3; their sum E more; the quotient and the product with it 3
    widest = far.amax(dim=1, keepdim=True)
    cp = (far + widest + E + 10) * U
    ep = cp * p + 2.0 ** -126
    el = (widest + E + 6) * U + 2 * U * (lse - top).abs() + U * lse.abs()
    f = counts[:E].double() / (n * k)
    bal, zl = E * (f * p.sum(dim=0)).sum() / n, (lse * lse).sum() / n
    eb = E * (f * (ep + (n + 4) * U * p).sum(dim=0)).sum() / n + 4 * U * bal
    ez = ((2 * lse.abs() * el + el * el) + (n + 4) * U * lse * lse).sum() / n
    losses = torch.stack([bal, zl])
    gb, gz = (float(v) for v in dlosses)
    dot = (p * f).sum(dim=1, keepdim=True)
    edot = ((ep + (E + 4) * U * p) * f).sum(dim=1, keepdim=True)
    inner = gb * E * (f - dot) + 2 * gz * lse
    einner = abs(gb) * E * (edot + 8 * U * (f + dot)) + 2 * abs(gz) * (el + 6 * U * lse.abs())
    v = p * inner / n
    d[keep] = v
    bd[keep] = (ep * (inner.abs() + einner) + p * einner) / n + 4 * U * v.abs()
    return (losses, torch.stack([eb, ez])), counts.int(), (d, rounded(d, bd, logits.dtype))


# ------------------------------------------------------------------- lora
def _pairs(t, dt, largest):
    """What a high and a low part leave of t; fp16's low part has no bits below 2^-25 of a
    largest value between 2^13 and 2^14."""
    e = E16[dt] ** 2 * t.abs() + 2.0 ** -149
    return e + (2.0 ** -38 * largest if dt == torch.float16 else 0.0)


def lora(x, a, b, ids, scale, base):
    """((t, bound), (y, bound)) row by row of the adapters."""
    R, K = x.shape
    n, rank, _ = a.shape
    dt = x.dtype
    t = torch.zeros(R, rank, dtype=torch.float64, device=x.device)
    et = torch.zeros_like(t)
    y = torch.zeros(R, b.shape[1], dtype=torch.float64, device=x.device) if base is None else base.double()
    ey = torch.zeros_like(y)
    for i in range(n):
        r = torch.nonzero(ids == i).flatten()
        if not r.numel():
            continue
        xr, A, B, s = x[r].double(), a[i].double(), b[i].double(), float(scale[i])
        t[r] = xr @ A.t()
        et[r] = (K + 2) * U * (xr.abs() @ A.abs().t())
        e = et[r] + _pairs(t[r], dt, (t[r].abs() + et[r]).amax(dim=1, keepdim=True))
        d = t[r] @ B.t()
        size = (t[r].abs() + e) @ B.abs().t()
        ey[r] = abs(s) * (e @ B.abs().t() + (2 * rank + 8) * U * size) + 2 * U * y[r].abs()
        y[r] = y[r] + s * d
    return (t, et), (y, rounded(y, ey, dt))


def lora_grads(dy, x, a, b, ids, scale, t, dx_base):
    """((dx, bound), (da, bound), (db, bound)) for the fp32 t that the forward call kept."""
    R, K = x.shape
    n, rank, _ = a.shape
    N, dt = b.shape[1], x.dtype
    dx = torch.zeros(R, K, dtype=torch.float64, device=x.device) if dx_base is None else dx_base.double()
    ex = torch.zeros_like(dx)
    da, db = torch.zeros(a.shape, dtype=torch.float64, device=x.device), torch.zeros(b.shape, dtype=torch.float64, device=x.device)
    ea, eb = torch.zeros_like(da), torch.zeros_like(db)
    for i in range(n):
        r = torch.nonzero(ids == i).flatten()
        if not r.numel():
            continue
        g, xr, A, B, s = dy[r].double(), x[r].double(), a[i].double(), b[i].double(), float(scale[i])
        M = r.numel()
        u = g @ B
        eu = (N + 2) * U * (g.abs() @ B.abs())
        e = eu + _pairs(u, dt, (u.abs() + eu).amax(dim=1, keepdim=True))
        size = (u.abs() + e) @ A.abs()
        ex[r] = abs(s) * (e @ A.abs() + (2 * rank + 8) * U * size) + 2 * U * dx[r].abs()
        dx[r] = dx[r] + s * (u @ A)
        # the parts' power of two is a segment's, at most all the adapter's rows
        e = eu + _pairs(u, dt, (u.abs() + eu).max())
        da[i] = s * (u.t() @ xr)
        ea[i] = abs(s) * (e.t() @ xr.abs() + (2 * M + 16) * U * ((u.abs() + e).t() @ xr.abs()))
        tr = t[r].double()
        e = _pairs(tr, dt, tr.abs().max())
        db[i] = s * (g.t() @ tr)
        eb[i] = abs(s) * (g.abs().t() @ e + (2 * M + 16) * U * (g.abs().t() @ (tr.abs() + e)))
    return (dx, rounded(dx, ex, dt)), (da, rounded(da, ea, dt)), (db, rounded(db, eb, dt))
