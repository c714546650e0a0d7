"""Operands and results whose byte and element offsets pass 32 bits, on whole
numbers (sums exact in any order, see tests/test_gpu_dense_exact_sums.py)."""
import pytest
import torch

from gpu_common import binding, log
from test_gpu_dense import BF, FP, IDS, gen
from test_gpu_dense_exact_sums import same, step, whole

pytestmark = pytest.mark.gpu

LD = 1 << 22          # the longest row stride


def spread(t):
    """The rows of t at the longest stride, 99 or NaN between them."""
    big = torch.full((t.shape[0], LD), 99 if t.dtype == torch.int8 else float("nan"), dtype=t.dtype, device="cuda")
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


@pytest.mark.parametrize("rows", [9, 600])
@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
def test_longest_strides(rows, dt):
    """600 rows: 5 GB of each 16-bit operand, 2.5 GB of codes."""
    log(f"case longest strides {rows} {dt}")
    B = binding()
    g = gen(rows)
    for H, I in ((264, 600), (131, 600)):                # read in place, and copied
        x, wg, wu = (whole(g, *s, dt=dt) for s in ((rows, H), (I, H), (I, H)))
        dh, gu, dg, du = step(g, rows, I, dt)
        xs, ws, us, es = (spread(t) for t in (x, wg, wu, dh))
        hs, dxs = spread(torch.zeros(rows, I, dtype=dt, device="cuda")), spread(torch.zeros(rows, H, dtype=dt, device="cuda"))
        h, kept = B.glu_forward(xs, ws, us, save=True, h=hs)
        h2, kept2 = B.glu_forward(x, wg, wu, save=True)
        same(kept[:, 0], (x.double() @ wg.double().t()).float(), "g")
        assert torch.equal(h, h2) and torch.equal(kept, kept2)
        dx, dwg, dwu = B.glu_backward(es, xs, ws, us, gu, dx=dxs)
        same(dx, (dg @ wg.double() + du @ wu.double()).float().to(dt), "dx")
        same(dwg, (dg.t() @ x.double()).float().to(dt), "dw_gate")
        same(dwu, (du.t() @ x.double()).float().to(dt), "dw_up")
        for t, n in ((hs, I), (dxs, H)):                 # nothing behind the rows was written
            assert torch.isnan(torch.as_strided(t, (rows, 64), (LD, 1), t.storage_offset() + n)).all()
        del xs, ws, us, es, hs, dxs
        q, w = whole(g, rows, H, dt=torch.int8, top=127), whole(g, I, H, dt=torch.int8, top=127)
        one, s = torch.ones(I, device="cuda"), torch.full((rows,), 2.0 ** -10, device="cuda")
        y = B.linear_i8(spread(q), spread(w), one, x_scale=s, out_dtype=dt)
        same(y, ((q.double() @ w.double().t()).float() * 2.0 ** -10).to(dt), "y")
        c, sc = B.quant_rows(spread(x))
        c2, sc2 = B.quant_rows(x)
        assert torch.equal(c, c2) and torch.equal(sc, sc2)


@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
def test_results_of_more_than_32_bits(dt):
    """2^20 rows of 1100: 2.3e9 elements (9.2 GB) of kept g and u, 4.8 GB of dg and du."""
    log(f"case long results {dt}")
    B = binding()
    M, H, I = 1 << 20, 16, 1100
    g = gen(1)
    x, wg, wu = (whole(g, *s, dt=dt) for s in ((M, H), (I, H), (I, H)))
    h, gu = B.glu_forward(x, wg, wu, save=True)
    for rows in (slice(0, 700), slice(M // 2 - 300, M // 2 + 300), slice(M - 700, M)):
        same(gu[rows, 0], (x[rows].double() @ wg.double().t()).float(), "g")
        same(gu[rows, 1], (x[rows].double() @ wu.double().t()).float(), "u")
        assert torch.equal(h[rows], B.glu_forward(x[rows], wg, wu))
    del h
    gu[:, 0] = 32
    dh = torch.zeros(M, I, dtype=dt, device="cuda")
    mark = torch.arange(0, M, 1021, device="cuda")       # rows that count, the last one among them
    mark[-1] = M - 1
    dh[mark] = whole(g, mark.numel(), I, dt=dt)
    dx, dwg, dwu = B.glu_backward(dh, x, wg, wu, gu)
    e, u, xm = dh[mark].double(), gu[mark, 1].double(), x[mark].double()
    dg, du = e * u, 32 * e
    want = torch.zeros(M, H, dtype=torch.float64, device="cuda")
    want[mark] = dg @ wg.double() + du @ wu.double()
    same(dx, want.float().to(dt), "dx")
    same(dwg, (dg.t() @ xm).float().to(dt), "dw_gate")
    same(dwu, (du.t() @ xm).float().to(dt), "dw_up")
    del dh, gu, dx
    q, w = whole(g, M, H, dt=torch.int8), whole(g, 2100, H, dt=torch.int8)
    y = B.linear_i8(q, w, torch.ones(2100, device="cuda"), x_scale=torch.ones(M, device="cuda"), out_dtype=dt)
    assert y.numel() > 2 ** 31
    for rows in (slice(0, 700), slice(M - 700, M)):
        same(y[rows], (q[rows].double() @ w.double().t()).float().to(dt), "y")
