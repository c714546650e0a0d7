"""Argument checks of the Python binding of the operators around the feed-forward
block, without a GPU: what would lose a gradient, and operands that do not fit."""
import pytest
import torch

from test_dense_binding import Operand

qr = pytest.importorskip("quantized_routed_expert_fp32_amd")
B = qr.binding
F, I32 = torch.float32, torch.int32


def t(*shape, dtype=torch.bfloat16, grad=False):
    return torch.ones(*shape, dtype=dtype).requires_grad_(grad)


def ids(*shape):
    return torch.zeros(*shape, dtype=I32)


HISTORY = {
    "norm_forward x": lambda g: B.norm_forward(t(2, 8, grad=g), t(8)),
    "norm_forward weight": lambda g: B.norm_forward(t(2, 8), t(8, grad=g)),
    "norm_forward residual": lambda g: B.norm_forward(t(2, 8), t(8), residual=t(2, 8, grad=g)),
    "norm_i8 x": lambda g: B.norm_i8(t(2, 8, grad=g), t(8)),
    "norm_i8 weight": lambda g: B.norm_i8(t(2, 8), t(8, grad=g)),
    "norm_i8 residual": lambda g: B.norm_i8(t(2, 8), t(8), residual=t(2, 8, grad=g)),
    "norm_backward dy": lambda g: B.norm_backward(t(2, 8, grad=g), t(2, 8), t(8), t(2, dtype=F)),
    "norm_backward dtotal": lambda g: B.norm_backward(t(2, 8), t(2, 8), t(8), t(2, dtype=F), dtotal=t(2, 8, grad=g)),
    "balance_forward logits": lambda g: B.balance_forward(t(2, 8, dtype=F, grad=g), ids(2, 2)),
    "balance_backward dlosses": lambda g: B.balance_backward(t(2, dtype=F, grad=g), t(2, 8, dtype=F), ids(9), 2),
    "lora_forward x": lambda g: B.lora_forward(t(2, 8, grad=g), t(1, 2, 8), t(1, 4, 2), ids(2), t(1, dtype=F)),
    "lora_forward a": lambda g: B.lora_forward(t(2, 8), t(1, 2, 8, grad=g), t(1, 4, 2), ids(2), t(1, dtype=F)),
    "lora_forward b": lambda g: B.lora_forward(t(2, 8), t(1, 2, 8), t(1, 4, 2, grad=g), ids(2), t(1, dtype=F)),
    "lora_forward scale": lambda g: B.lora_forward(t(2, 8), t(1, 2, 8), t(1, 4, 2), ids(2), t(1, dtype=F, grad=g), save=True),
    "lora_forward base": lambda g: B.lora_forward(t(2, 8), t(1, 2, 8), t(1, 4, 2), ids(2), t(1, dtype=F), base=t(2, 4, grad=g)),
    "lora_backward dy": lambda g: B.lora_backward(t(2, 4, grad=g), t(2, 8), t(1, 2, 8), t(1, 4, 2), ids(2), t(1, dtype=F),
                                                  need_dw=False),
    "lora_backward dx_base": lambda g: B.lora_backward(t(2, 4), t(2, 8), t(1, 2, 8), t(1, 4, 2), ids(2), t(1, dtype=F),
                                                       dx_base=t(2, 8, grad=g), need_dw=False),
}


@pytest.mark.parametrize("name", HISTORY)
def test_operands_that_want_a_gradient_are_refused(name):
    fn, arg = name.split()
    with pytest.raises(B.MoeError, match=f"{fn}: {arg} requires a gradient"):
        HISTORY[name](True)
    with torch.no_grad(), pytest.raises(B.MoeError, match="needs device memory"):
        HISTORY[name](True)
    with pytest.raises(B.MoeError, match="needs device memory"):
        HISTORY[name](False)


def test_calls_of_a_training_step_take_parameters():
    p = lambda *s, dtype=torch.bfloat16: torch.nn.Parameter(torch.ones(*s, dtype=dtype))
    for f in (lambda: B.norm_forward(p(2, 8), p(8), residual=p(2, 8), save=True),
              lambda: B.norm_forward(p(2, 8), p(8), rstd=t(2, dtype=F)),
              lambda: B.norm_backward(t(2, 8), p(2, 8), p(8), t(2, dtype=F)),
              lambda: B.balance_forward(p(2, 8, dtype=F), ids(2, 2), save=True),
              lambda: B.balance_backward(t(2, dtype=F), p(2, 8, dtype=F), ids(9), 2),
              lambda: B.lora_forward(p(2, 8), p(1, 2, 8), p(1, 4, 2), ids(2), t(1, dtype=F), base=p(2, 4), save=True),
              lambda: B.lora_backward(t(2, 4), p(2, 8), p(1, 2, 8), p(1, 4, 2), ids(2), t(1, dtype=F), need_dw=False)):
        with pytest.raises(B.MoeError, match="needs device memory"):
            f()


class Dev(Operand):
    """A device tensor's attributes of any number of dimensions."""

    def __init__(self, *shape, dtype=torch.bfloat16, stride=None, dev=0, grad=False):
        c = [1]
        for n in reversed(shape[1:]):
            c.insert(0, c[0] * n)
        super().__init__(*shape, dtype=dtype, stride=tuple(c) if stride is None else stride)
        self.dev, self.requires_grad, self.device = dev, grad, f"cuda:{dev}"

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        c = 1
        for n, s in zip(reversed(self.shape), reversed(self._stride)):
            if n > 1 and s != c:
                return False
            c *= n
        return True


BF, FP = torch.bfloat16, torch.float16
NORM = dict(x=Dev(4, 8), weight=Dev(8))
LORA = dict(x=Dev(4, 8), a=Dev(3, 2, 8), b=Dev(3, 6, 2), ids=Dev(4, dtype=I32), scale=Dev(3, dtype=F))

BAD = [
    (lambda: B.norm_forward(**{**NORM, "x": Dev(8)}), "x: 1-D"),
    (lambda: B.norm_forward(**{**NORM, "x": Dev(4, 8, dtype=F)}), "dtype torch.float32"),
    (lambda: B.norm_forward(**{**NORM, "x": Dev(4, 8, dtype=FP)}, residual=Dev(4, 8)), "x: dtype torch.float16"),
    (lambda: B.norm_forward(**{**NORM, "x": Dev(4, 8, dtype=F)}, residual=Dev(4, 8, dtype=F)), "residual: dtype"),
    (lambda: B.norm_forward(**NORM, residual=Dev(4, 7)), "residual: shape"),
    (lambda: B.norm_forward(**NORM, residual=Dev(4, 8, dev=1)), "residual: on cuda:1"),
    (lambda: B.norm_forward(**{**NORM, "weight": Dev(7)}), "weight"),
    (lambda: B.norm_forward(**{**NORM, "weight": Dev(8, dtype=FP)}), "weight"),
    (lambda: B.norm_forward(**{**NORM, "x": Dev(4, 8, stride=(1, 4))}), "x: the elements of a row"),
    (lambda: B.norm_forward(**{**NORM, "x": Dev(2 ** 31, 8)}), "x: shape"),
    (lambda: B.norm_backward(Dev(4, 7), Dev(4, 8), Dev(8), Dev(4, dtype=F)), "dy: shape"),
    (lambda: B.norm_backward(Dev(4, 8), Dev(4, 8), Dev(8), Dev(5, dtype=F)), "rstd"),
    (lambda: B.norm_backward(Dev(4, 8), Dev(4, 8), Dev(8), None), "rstd: needed"),
    (lambda: B.norm_backward(Dev(4, 8), Dev(4, 8), Dev(8), Dev(4, dtype=F), need_dx=False, need_dw=False), "neither"),
    (lambda: B.norm_backward(Dev(4, 8), Dev(4, 8), Dev(8), Dev(4, dtype=F), dtotal=Dev(4, 8), need_dx=False), "dtotal"),
    (lambda: B.balance_forward(Dev(4, 8, dtype=I32), Dev(4, 2, dtype=I32)), "logits: dtype"),
    (lambda: B.balance_forward(Dev(4, 8, dtype=F), Dev(4, 2, dtype=torch.int64)), "ids: dtype"),
    (lambda: B.balance_forward(Dev(4, 8, dtype=F), Dev(5, 2, dtype=I32)), "ids: shape"),
    (lambda: B.balance_forward(Dev(4, 8, dtype=F), Dev(4, 2, dtype=I32, stride=(3, 1))), "ids: needs contiguous"),
    (lambda: B.balance_forward(Dev(4, 8, dtype=F), Dev(4, 2, dtype=I32), mask=Dev(4, dtype=F)), "mask"),
    (lambda: B.balance_forward(Dev(4, 8, dtype=F), Dev(4, 2, dtype=I32), mask=Dev(5, dtype=torch.bool)), "mask"),
    (lambda: B.balance_backward(Dev(2, dtype=F), Dev(4, 8, dtype=F), Dev(8, dtype=I32), 2), "counts"),
    (lambda: B.balance_backward(Dev(1, dtype=F), Dev(4, 8, dtype=F), Dev(9, dtype=I32), 2), "dlosses"),
    (lambda: B.balance_backward(None, Dev(4, 8, dtype=F), Dev(9, dtype=I32), 2), "both needed"),
    (lambda: B.lora_forward(**{**LORA, "x": Dev(4, 9)}), "x: rows of 9"),
    (lambda: B.lora_forward(**{**LORA, "a": Dev(2, 8)}), "a: 2-D"),
    (lambda: B.lora_forward(**{**LORA, "b": Dev(2, 6, 2)}), "b: shape"),
    (lambda: B.lora_forward(**{**LORA, "b": Dev(6, 2)}), "b: 2-D"),
    (lambda: B.lora_forward(**{**LORA, "b": Dev(3, 6, 3)}), "b: shape"),
    (lambda: B.lora_forward(**{**LORA, "a": Dev(3, 2, 8, dtype=FP)}), "a: dtype"),
    (lambda: B.lora_forward(**{**LORA, "a": Dev(3, 2, 8, stride=(16, 1, 2))}), "a: the elements of a row"),
    (lambda: B.lora_forward(**{**LORA, "a": Dev(2 ** 31, 2, 8)}), "a: shape"),
    (lambda: B.lora_forward(**{**LORA, "ids": Dev(4, dtype=torch.int64)}), "ids"),
    (lambda: B.lora_forward(**{**LORA, "ids": None}), "ids, scale"),
    (lambda: B.lora_forward(**{**LORA, "scale": Dev(4, dtype=F)}), "scale"),
    (lambda: B.lora_forward(**{**LORA, "scale": Dev(3, dtype=F, dev=1)}), "scale: on cuda:1"),
    (lambda: B.lora_backward(Dev(4, 5), **LORA, need_dw=False), "dy: shape"),
    (lambda: B.lora_backward(Dev(4, 6), **LORA), "t: needed"),
    (lambda: B.lora_backward(Dev(4, 6), **LORA, t=Dev(4, 3, dtype=F)), "t: shape"),
    (lambda: B.lora_backward(Dev(4, 6), **LORA, t=Dev(4, 2, dtype=F, stride=(5, 1))), "t: needs contiguous"),
    (lambda: B.lora_backward(Dev(4, 6), **LORA, need_dx=False, need_dw=False), "neither"),
    (lambda: B.lora_backward(Dev(4, 6), **LORA, need_dx=False, t=Dev(4, 2, dtype=F), dx_base=Dev(4, 8)), "dx_base"),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_operands_that_do_not_fit(i):
    call, msg = BAD[i]
    with pytest.raises(B.MoeError, match=msg):
        call()
