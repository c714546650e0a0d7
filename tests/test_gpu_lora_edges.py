"""Low-rank adapters where a value is not finite: whom it reaches, and whom it does not."""
import pytest
import torch

from gpu_common import binding, log
from test_gpu_lora import BF, FP, IDS, problem, rnd

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
@pytest.mark.parametrize("R,rank", [(6, 4), (300, 20), (300, 70), (1500, 8)])
def test_unused_adapters_have_zero_gradients_whatever_their_scale(R, rank, dt):
    """A slot of a pool that no row is on may hold anything, its scale too."""
    log(f"case lora unused scale {R} {rank} {dt}")
    B = binding()
    p, g = problem(R + rank, R, 136, 72, rank, 4, dt, "any")
    p["ids"] = torch.where(p["ids"] == 2, -1, p["ids"])
    dy = rnd(g, R, 72, dt=dt)
    y, t = B.lora_forward(**p, save=True)
    want = B.lora_backward(dy, **p, t=t)
    for v in (NAN, INF, -INF):
        q = dict(p, scale=p["scale"].clone())
        q["scale"][2] = v
        y2, t2 = B.lora_forward(**q, save=True)
        assert torch.equal(y2, y) and torch.equal(t2, t)
        got = B.lora_backward(dy, **q, t=t)
        assert (got[1][2] == 0).all() and (got[2][2] == 0).all(), v
        assert all(torch.equal(a, b) for a, b in zip(got, want)), v


# one step of the rank (up to 64) and several, rows of one adapter and of many
@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
@pytest.mark.parametrize("kind", ["one", "any"])
@pytest.mark.parametrize("rank", [16, 64, 65, 129, 256])
def test_rows_that_are_not_finite_leave_the_others_bits(rank, kind, dt):
    log(f"case lora rows not finite {rank} {kind} {dt}")
    B, R = binding(), 300
    p, g = problem(rank, R, 264, 200, rank, 3, dt, kind)
    base, dy, dxb = rnd(g, R, 200, dt=dt), rnd(g, R, 200, dt=dt), rnd(g, R, 264, dt=dt)
    y, t = B.lora_forward(**p, base=base, save=True)
    dx = B.lora_backward(dy, **p, dx_base=dxb, need_dw=False)[0]
    bad = [1, 2, 3, 70, 255]

    def spoil(v):
        v = v.clone()
        v[1], v[2, 5], v[3], v[70, 7], v[255] = NAN, INF, torch.finfo(dt).max, -INF, -torch.finfo(dt).max
        return v

    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[bad] = False
    y2, t2 = B.lora_forward(**dict(p, x=spoil(p["x"])), base=base, save=True)
    assert torch.equal(y2[keep], y[keep]) and torch.equal(t2[keep], t[keep])
    dx2 = B.lora_backward(spoil(dy), **p, dx_base=dxb, need_dw=False)[0]
    assert torch.equal(dx2[keep], dx[keep])
    on = p["ids"][1] >= 0
    assert not on or (y2[1].isnan().all() and dx2[1].isnan().all())


@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
@pytest.mark.parametrize("rank", [16, 64, 65, 129, 256])
def test_infinite_weights_give_infinity_and_leave_the_other_columns_bits(rank, dt):
    log(f"case lora infinite weights {rank} {dt}")
    B, R = binding(), 200
    p, g = problem(rank + 1, R, 136, 72, rank, 1, dt, "one")
    j = rank - 1
    y, t = B.lora_forward(**p, save=True)
    dy = rnd(g, R, 72, dt=dt)
    dx = B.lora_backward(dy, **p, need_dw=False)[0]
    u = dy.double() @ p["b"][0].double()
    q = dict(p, b=p["b"].clone())
    q["b"][0, 7, j] = INF
    y2 = B.lora_forward(**q)
    assert (t[:, j] != 0).all()
    assert torch.equal(y2[:, 7].double(), torch.sign(t[:, j]).double() * INF)
    other = torch.arange(72, device="cuda") != 7
    assert torch.equal(y2[:, other], y[:, other])
    q = dict(p, a=p["a"].clone())
    q["a"][0, j, 9] = -INF
    dx2 = B.lora_backward(dy, **q, need_dw=False)[0]
    # where fp32 sums leave no doubt of u's sign
    sure = u[:, j].abs() > 1e-3
    assert sure.sum() > R / 2 and torch.equal(dx2[sure, 9].double(), -torch.sign(u[sure, j]) * INF)
    other = torch.arange(136, device="cuda") != 9
    assert torch.equal(dx2[:, other], dx[:, other])
