"""dx in the place of dy, which da and db still read: refused with them, right without."""
import pytest
import torch

from gpu_common import binding, log
from test_gpu_lora import BF, problem, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [5, 300])
def test_dx_in_the_place_of_dy_or_x(R):
    log(f"case lora dx over dy {R}")
    B = binding()
    p, g = problem(R, R, 136, 136, 12, 3, BF, "any")
    dy = rnd(g, R, 136, dt=BF)
    _, t = B.lora_forward(**p, save=True)
    want = B.lora_backward(dy, **p, dx_base=dy, need_dw=False)[0]
    z, x = dy.clone(), p["x"].clone()
    for kw in (dict(dx=z), dict(dx=z, dx_base=z), dict(dx=p["x"]), dict(dx=p["x"], dx_base=z)):
        with pytest.raises(B.MoeError, match="which da and db are computed from"):
            B.lora_backward(z, **p, t=t, **kw)
    assert torch.equal(z, dy) and torch.equal(p["x"], x)
    assert B.lora_backward(z, **p, dx_base=z, dx=z, need_dw=False)[0] is z and torch.equal(z, want)
