"""Sizes at which a workgroup of the operators around the feed-forward block takes
several rows, or several steps of columns, one behind the other."""
import pytest
import torch

import test_gpu_balance as balance
import test_gpu_lora as lora
import test_gpu_norm as norm
from gpu_common import binding, log

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
IDS = {BF: "bf16", FP: "fp16", F32: "fp32"}

# 8192 waves of a forward call and 4096 of the gradients take a row each: more rows than that
# in rows of 64, 128, 256 and 512 threads, and of 1024 threads with one, two and eight chunks each
NORM = [(8200, 64), (8195, 511), (4100, 520), (2060, 1288), (1030, 2060), (520, 4104), (520, 9000), (520, 20000), (515, 16390)]


@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
@pytest.mark.parametrize("R,H", NORM)
def test_norm(R, H, dt):
    log(f"case rows norm {R} {H} {dt}")
    B, g = binding(), norm.gen(R + H)
    w = (1.0 + norm.rnd(g, H, std=0.3)).to(dt)
    norm.check(B, norm.rnd(g, R, H, dt=dt), w, None, dt)
    norm.check(B, norm.rnd(g, R, H), w, norm.rnd(g, R, H, dt=dt), dt)


@pytest.mark.parametrize("R,H", NORM)
def test_norm_total_in_place(R, H):
    log(f"case rows norm in place {R} {H}")
    B, g = binding(), norm.gen(H)
    x, res, w = norm.rnd(g, R, H, dt=BF), norm.rnd(g, R, H, dt=BF), norm.rnd(g, H, dt=BF)
    y, total, _ = B.norm_forward(x, w, residual=res)
    assert torch.equal(total, x + res)
    for into in (0, 1):
        xx, rr = x.clone(), res.clone()
        t = (xx, rr)[into]
        got = B.norm_forward(xx, w, residual=rr, total=t)[0]
        assert torch.equal(got, y) and torch.equal(t, total)


@pytest.mark.parametrize("R,H", NORM)
def test_norm_rows_that_are_not_finite_leave_the_others_bits(R, H):
    """Rows that one workgroup takes behind one another share its LDS and registers, not their values."""
    log(f"case rows norm not finite {R} {H}")
    B, g = binding(), norm.gen(H + 1)
    x, w, dy = norm.rnd(g, R, H, dt=BF), norm.rnd(g, H, dt=BF), norm.rnd(g, R, H, dt=BF)
    y, _, rstd = B.norm_forward(x, w, save=True)
    q, scale, _, _ = B.norm_i8(x, w)
    dx = B.norm_backward(dy, x, w, rstd, need_dw=False)[0]
    x2 = x.clone()
    x2[1], x2[R // 2, H // 2], x2[R // 3] = float("nan"), float("inf"), torch.finfo(BF).max
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[[1, R // 2, R // 3]] = False
    y2, _, rstd2 = B.norm_forward(x2, w, save=True)
    q2, scale2, _, _ = B.norm_i8(x2, w)
    dx2 = B.norm_backward(dy, x2, w, rstd2, need_dw=False)[0]
    for a, b in ((y2, y), (rstd2, rstd), (q2, q), (scale2, scale), (dx2, dx)):
        assert torch.equal(a[keep], b[keep])


# over 2048 workgroups of 16 rows (up to 256 experts) or of 4
@pytest.mark.parametrize("dt", [F32, BF, FP], ids=IDS.get)
@pytest.mark.parametrize("R,E,k", [(33000, 256, 8), (33000, 60, 2), (8300, 300, 4)])
def test_balance(R, E, k, dt):
    log(f"case rows balance {R} {E} {dt}")
    balance.check(binding(), *balance.inputs(R + E, R, E, k, dt, 0.2))


# 64 tiles of rows: three steps of 64 columns a workgroup, the last one ragged
@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
@pytest.mark.parametrize("rank", [16, 64, 100])
def test_lora(rank, dt):
    log(f"case rows lora {rank} {dt}")
    B, R, K_, N = binding(), 4096, 2060, 2105
    p, g = lora.problem(rank, R, K_, N, rank, 3, dt, "runs")
    lora.check(B, p, g)
    base, dy, dxb = lora.rnd(g, R, N, dt=dt), lora.rnd(g, R, N, dt=dt), lora.rnd(g, R, K_, dt=dt)
    y = B.lora_forward(**p, base=base)
    z = base.clone()
    assert B.lora_forward(**p, base=z, y=z) is z and torch.equal(z, y)
    dx = B.lora_backward(dy, **p, dx_base=dxb, need_dw=False)[0]
    z = dxb.clone()
    B.lora_backward(dy, **p, dx_base=z, dx=z, need_dw=False)
    assert torch.equal(z, dx)
