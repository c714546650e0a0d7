"""The dense operators record no history: a call whose result would silently
lack one is refused, wherever its operands live (so this needs no GPU)."""
import pytest
import torch

qr = pytest.importorskip("quantized_routed_expert_fp32_amd")
B = qr.binding


def t(*shape, dtype=torch.bfloat16, grad=False):
    return torch.ones(*shape, dtype=dtype).requires_grad_(grad)


def i8(*shape):
    return torch.ones(*shape, dtype=torch.int8)


F = torch.float32
CALLS = {
    "glu_forward x": lambda g: B.glu_forward(t(2, 8, grad=g), t(4, 8), t(4, 8)),
    "glu_forward w_gate": lambda g: B.glu_forward(t(2, 8), t(4, 8, grad=g), t(4, 8)),
    "glu_forward w_up": lambda g: B.glu_forward(t(2, 8), t(4, 8), t(4, 8, grad=g)),
    "glu_backward dh": lambda g: B.glu_backward(t(2, 4, grad=g), t(2, 8), t(4, 8), t(4, 8), t(2, 2, 4, dtype=F)),
    "glu_i8 x": lambda g: B.glu_i8(t(2, 8, grad=g), i8(4, 8), t(4, dtype=F), i8(4, 8), t(4, dtype=F)),
    "glu_i8 s_up": lambda g: B.glu_i8(t(2, 8), i8(4, 8), t(4, dtype=F), i8(4, 8), t(4, dtype=F, grad=g)),
    "linear_i8 x": lambda g: B.linear_i8(t(2, 8, grad=g), i8(4, 8), t(4, dtype=F)),
    "linear_i8 s_w": lambda g: B.linear_i8(t(2, 8), i8(4, 8), t(4, dtype=F, grad=g)),
    "linear_i8 bias": lambda g: B.linear_i8(t(2, 8), i8(4, 8), t(4, dtype=F), bias=t(4, dtype=F, grad=g)),
    "linear_i8 x_scale": lambda g: B.linear_i8(i8(2, 8), i8(4, 8), t(4, dtype=F), x_scale=t(2, dtype=F, grad=g)),
}


@pytest.mark.parametrize("name", CALLS)
def test_operands_that_want_a_gradient_are_refused(name):
    fn, arg = name.split()
    with pytest.raises(B.MoeError, match=f"{fn}: {arg} requires a gradient"):
        CALLS[name](True)
    # without history asked for, the call goes on (here to the check of the device)
    with torch.no_grad(), pytest.raises(B.MoeError, match="needs device memory"):
        CALLS[name](True)
    with pytest.raises(B.MoeError, match="needs device memory"):
        CALLS[name](False)


def test_calls_of_a_training_step_take_parameters():
    """save=True says that the caller runs glu_backward; parameters are its operands too."""
    p = lambda *s: torch.nn.Parameter(torch.ones(*s, dtype=torch.bfloat16))
    for f in (lambda: B.glu_forward(p(2, 8), p(4, 8), p(4, 8), save=True),
              lambda: B.glu_forward(p(2, 8), p(4, 8), p(4, 8), gu=t(2, 2, 4, dtype=F)),
              lambda: B.glu_backward(t(2, 4), p(2, 8), p(4, 8), p(4, 8), t(2, 2, 4, dtype=F)),
              lambda: B.quant_rows(p(4, 8))):
        with pytest.raises(B.MoeError, match="needs device memory"):
            f()
