"""The balance losses' sums over rows, and probabilities below the normal numbers, on
logits whose every other rounding is known."""
import math

import pytest
import torch

import block_common as K
from gpu_common import binding, log

pytestmark = pytest.mark.gpu
U = K.U
ROWS = [1, 64, 200, 257, 3000, 20000, 70000]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("R", ROWS)
def test_z_loss_sums_in_64_bits(R, masked):
    """One expert: its logsumexp is the logit itself, without rounding, and its square has 48
    bits. Sums in 64 bits are good to R 2^-53, so the result is off by its own rounding alone."""
    log(f"case balance z sums {R} {masked}")
    B = binding()
    for seed in range(6):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        l = 3.0 + torch.rand(R, 1, generator=g, device="cuda")
        mask = torch.rand(R, generator=g, device="cuda") < 0.9 if masked else None
        ids = torch.zeros(R, 1, dtype=torch.int32, device="cuda")
        losses, counts = B.balance_forward(l, ids, mask=mask)
        kept = l if mask is None else l[mask]
        n = kept.shape[0]
        assert int(counts[1]) == n
        want = (kept.double() ** 2).mean().item() if n else 0.0
        assert abs(losses[1].item() - want) <= U * want * (1 + 1e-6), seed
        assert losses[0].item() == (1.0 if n else 0.0)


@pytest.mark.parametrize("E", [8, 64, 200, 300])
@pytest.mark.parametrize("R", ROWS)
def test_balance_loss_sums(R, E):
    """Rows of m equal logits, the others -inf: every probability is fp32(1 / m). A thread adds its
    few rows in fp32, and its workgroup's sum is rounded to fp32: the rest is in 64 bits."""
    log(f"case balance sums {R} {E}")
    B = binding()
    g = torch.Generator(device="cuda")
    g.manual_seed(R + E)
    m = torch.randint(2, E + 1, (R, 1), generator=g, device="cuda")
    on = torch.rand(R, E, generator=g, device="cuda").argsort(dim=1).argsort(dim=1) < m
    l = torch.where(on, 0.0, -math.inf)
    ids = on.float().topk(2, dim=1).indices.to(torch.int32)
    losses, counts = B.balance_forward(l, ids)
    p = torch.where(on, (1.0 / m.float()).double(), 0.0)
    c = torch.bincount(ids.flatten().long(), minlength=E)
    assert torch.equal(counts[:E].long(), c)
    want = E * (c.double() * p.sum(dim=0)).sum().item() / (R * R * 2)
    groups = 32 if E <= 256 else 8                     # rows that a workgroup takes at a time
    parts = 1 if R <= 256 else min(-(-R // 32), 256)
    adds = -(-(-(-R // parts)) // groups)
    assert abs(losses[0].item() - want) <= (adds + 2) * U * want


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("E", [5, 64, 300])
def test_probabilities_below_the_normal_numbers(E, dt):
    """e^-88 and e^-96 are subnormal in fp32, and count: their gradients are normal numbers where the
    z loss weighs much. The exponential and its product with 1 / z round to 2^-149 each."""
    log(f"case balance subnormal {E} {dt}")
    B = binding()
    R = 40
    l = torch.full((R, E), -math.inf, device="cuda")
    l[:, 0], l[:, 1], l[:, 2], l[:, 3] = 1024.0, 1024.0 - 88.0, 1024.0 - 96.0, 1024.0 - 85.0
    l = l.to(dt)
    ids = torch.zeros(R, 1, dtype=torch.int32, device="cuda")
    losses, counts = B.balance_forward(l, ids)
    assert losses[1].item() == 2.0 ** 20
    d = torch.tensor([0.0, 1e6], device="cuda")
    got = B.balance_backward(d, l, counts, 1)
    for c in (1, 2, 3):
        far = 1024.0 - l[0, c].item()                  # (939 is 940 in bf16)
        p = math.exp(-far)
        factor = 2 * 1e6 * 1024.0 / R
        want = torch.full((R,), p * factor, dtype=torch.float64)
        bound = torch.full((R,), ((far + 10) * U * p + 2 * 2.0 ** -149) * factor, dtype=torch.float64)
        K.close(got[:, c], want, K.rounded(want, bound, dt), f"dlogits {far}")
    assert (got[:, 4:] == 0).all()
