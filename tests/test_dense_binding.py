"""Argument checks of the dense operators' Python binding that need no GPU: the
operands are stand-ins with a tensor's attributes, nothing is allocated or run."""
import pytest
import torch

qr = pytest.importorskip("quantized_routed_expert_fp32_amd")
B = qr.binding


class Operand:
    """A device tensor's attributes, without its memory."""
    is_cuda = True
    requires_grad = False

    def __init__(self, *shape, dtype=torch.bfloat16, stride=None):
        self.shape, self.dtype = shape, dtype
        self._stride = stride if stride is not None else (shape[1], 1)

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self._stride

    def get_device(self):
        return 0

    def data_ptr(self):
        return 1 << 20


BIG = [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 33 + 64]


@pytest.mark.parametrize("n", BIG)
def test_sizes_that_do_not_fit_the_argument_block(n):
    """The argument blocks hold 32 bits: more rows or columns are refused, not cut off."""
    w = Operand(32, 8)
    q, qw = Operand(4, 8, dtype=torch.int8), Operand(32, 8, dtype=torch.int8)
    with pytest.raises(B.MoeError, match="x: shape"):
        B._glu_args(Operand(n, 8), w, w, "silu")
    with pytest.raises(B.MoeError, match="x: shape"):
        B._glu_args(Operand(4, n), w, w, "silu")
    with pytest.raises(B.MoeError, match="w_gate: shape"):
        B._glu_args(Operand(4, 8), Operand(n, 8), Operand(n, 8), "silu")
    with pytest.raises(B.MoeError, match="x: shape"):
        B._linear_args(Operand(n, 8), qw, Operand(32, dtype=torch.float32, stride=(1,)), None, None, None)
    with pytest.raises(B.MoeError, match="w: shape"):
        B._linear_args(q, Operand(n, 8, dtype=torch.int8), None, None, Operand(4, dtype=torch.float32, stride=(1,)), None)
    with pytest.raises(B.MoeError, match="x: shape"):
        B.quant_rows(Operand(n, 8, dtype=torch.float32))


def test_sizes_that_fit():
    w = Operand(32, 8)
    a, dt, dev = B._glu_args(Operand(2 ** 31 - 1, 8), w, w, "silu")
    assert (a.rows, a.hidden, a.inter, a.ldx, dt, dev) == (2 ** 31 - 1, 8, 32, 8, torch.bfloat16, 0)
