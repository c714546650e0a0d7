"""Workspaces of exactly the size that is asked for, among bytes that must stay as they are."""
import pytest
import torch

from gpu_common import binding, log
from test_gpu_balance import inputs
from test_gpu_lora import BF, FP, gen, problem, rnd

pytestmark = pytest.mark.gpu
GUARD = 1 << 20


def guarded(n):
    """(workspace of n bytes, check that what lies before and behind it is untouched)"""
    buf = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    assert buf.data_ptr() % 256 == 0

    def untouched():
        return bool((buf[:GUARD] == 0xA5).all() and (buf[GUARD + n:] == 0xA5).all())

    return buf[GUARD:GUARD + n], untouched


# one sorting workgroup and several, ranges of K, adapters of several segments, ranks of several steps
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("kind", ["any", "one"])
@pytest.mark.parametrize("R,K_,N,rank,n", [(65, 64, 64, 8, 1), (500, 200, 264, 16, 5), (700, 1283, 769, 20, 3), (8193, 72, 40, 8, 300),
                                           (9000, 136, 72, 100, 2), (3000, 520, 1030, 256, 7), (70, 4104, 40, 65, 1000)])
def test_lora(R, K_, N, rank, n, kind, dt):
    log(f"case workspace lora {R} {K_} {N} {rank} {n} {kind} {dt}")
    B = binding()
    p, g = problem(R + rank, R, K_, N, rank, n, dt, kind)
    dy = rnd(g, R, N, dt=dt)
    want = B.lora_forward(**p, save=True)
    ws, untouched = guarded(B.lora_workspace_size(**p))
    got = B.lora_forward(**p, save=True, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and untouched()
    grads = B.lora_backward(dy, **p, t=want[1])
    ws, untouched = guarded(B.lora_workspace_size(**p, kind=B.MOE_LORA_BACKWARD))
    got = B.lora_backward(dy, **p, t=want[1], ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, grads)) and untouched()


@pytest.mark.parametrize("R,H", [(1, 1), (5, 77), (1100, 1283), (4200, 64), (300, 9001), (260, 65536)])
def test_norm(R, H):
    log(f"case workspace norm {R} {H}")
    B, g = binding(), gen(R + H)
    x, w, dy = rnd(g, R, H, dt=BF), rnd(g, H, dt=BF), rnd(g, R, H, dt=BF)
    rstd = B.norm_forward(x, w, save=True)[2]
    want = B.norm_backward(dy, x, w, rstd)
    ws, untouched = guarded(B.norm_backward_workspace_size(x, w))
    got = B.norm_backward(dy, x, w, rstd, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and untouched()


@pytest.mark.parametrize("R,E", [(1, 1), (64, 64), (257, 7), (9000, 257), (20000, 1024)])
def test_balance(R, E):
    log(f"case workspace balance {R} {E}")
    B = binding()
    l, ids, mask, _ = inputs(R + E, R, E, 1, torch.float32, 0.2)
    want = B.balance_forward(l, ids, mask=mask)
    ws, untouched = guarded(B.balance_workspace_size(R, E))
    got = B.balance_forward(l, ids, mask=mask, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and untouched()
