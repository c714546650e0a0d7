"""8-bit codes of values next to the borders between two codes, on either side
of what the quantiser's fp32 product tells apart. The border of codes n and n +
1 is s (n + 1/2), which is exact in 64 bits, so that the oracle needs no division.
"""
import pytest
import torch

from gpu_common import binding, log
from test_gpu_dense import BF, FP, gen

pytestmark = pytest.mark.gpu


def codes(x, s):
    """Half-even codes of rows x by their borders (s > 0)."""
    x, s = x.double(), s.double()[:, None]
    n = torch.floor(x / s)                               # off by one at most: put right below
    n = torch.where(x < n * s, n - 1, torch.where(x >= (n + 1) * s, n + 1, n))
    border = (n + 0.5) * s
    q = torch.where(x > border, n + 1, torch.where(x < border, n, n + n.remainder(2)))
    return q.clamp(-127, 127).to(torch.int8)


def scale(m):
    """fp32(m / 127), on the CPU (on the device torch multiplies by a reciprocal)."""
    return (m.float().cpu() / torch.tensor(127.0)).cuda()


@pytest.mark.parametrize("power", [0, -90, 100, -120])
def test_values_next_to_a_border(power):
    log(f"case borders {power}")
    B = binding()
    R = 300
    m = torch.ldexp(1 + torch.rand(R, generator=gen(power), device="cuda"), torch.tensor(power, device="cuda"))
    s = scale(m)
    n = torch.arange(-127, 127, device="cuda").double() + 0.5
    x = (n * s.double()[:, None]).float()
    x = torch.cat([(x.view(torch.int32) + u).view(torch.float32) for u in range(-4, 5)] + [m[:, None]], dim=1)
    q, got = B.quant_rows(x.contiguous())
    assert torch.equal(got, s)
    assert torch.equal(q, codes(x, s))
    assert (q[:, -1] == 127).all()


@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
def test_halves_of_the_largest_value(dt):
    """x = m / 2 is 63.5 s but for the rounding of s, 2^-24 at most: the code is
    63 or 64 by that alone (64 on the tie). Through quant_rows and the decode
    form's own quantiser."""
    B = binding()
    bits = 7 if dt == BF else 10
    m = 1 + torch.arange(2 ** bits, device="cuda").float() / 2 ** bits
    x = torch.stack([m, m / 2, -m / 2, m / 4, -m], dim=1).to(dt).contiguous()
    s = scale(x[:, 0])
    want = codes(x, s)
    assert (want[:, 1] == 63).any() and (want[:, 1] == 64).any()
    q, got = B.quant_rows(x)
    assert torch.equal(got, s) and torch.equal(q, want)
    w = torch.zeros(5, 5, dtype=torch.int8, device="cuda")
    w.fill_diagonal_(1)                                  # one code each
    one = torch.ones(5, device="cuda")
    for first in range(0, x.shape[0], 16):
        rows = slice(first, first + 16)
        assert torch.equal(B.linear_i8(x[rows], w, one), B.linear_i8(want[rows], w, one, x_scale=s[rows], out_dtype=dt))
