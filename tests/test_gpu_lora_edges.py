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
