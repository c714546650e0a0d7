"""Tangents of forward-mode differentiation: the operators would drop them without a
word, so an operand that carries one is refused, also under no_grad (which leaves that mode on)."""
import pytest
import torch
from torch.autograd import forward_ad as fwd

qr = pytest.importorskip("quantized_routed_expert_fp32_amd")
B = qr.binding
F, I32 = torch.float32, torch.int32


def t(*shape, dtype=torch.bfloat16):
    return torch.ones(*shape, dtype=dtype)


def i8(*shape):
    return torch.ones(*shape, dtype=torch.int8)


LORA = dict(x=t(2, 8), a=t(1, 2, 8), b=t(1, 4, 2), ids=torch.zeros(2, dtype=I32), scale=t(1, dtype=F))
# function, its operands that have a gradient, the others
CALLS = [
    ("glu_forward", dict(x=t(2, 8), w_gate=t(4, 8), w_up=t(4, 8)), {}),
    ("glu_forward", dict(x=t(2, 8), w_gate=t(4, 8), w_up=t(4, 8)), dict(save=True)),
    ("glu_backward", dict(dh=t(2, 4), x=t(2, 8), w_gate=t(4, 8), w_up=t(4, 8), gu=t(2, 2, 4, dtype=F)), {}),
    ("glu_i8", dict(x=t(2, 8), s_gate=t(4, dtype=F), s_up=t(4, dtype=F)), dict(w_gate=i8(4, 8), w_up=i8(4, 8))),
    ("linear_i8", dict(x=t(2, 8), s_w=t(4, dtype=F), bias=t(4, dtype=F)), dict(w=i8(4, 8))),
    ("linear_i8", dict(x_scale=t(2, dtype=F)), dict(x=i8(2, 8), w=i8(4, 8), s_w=t(4, dtype=F))),
    ("norm_forward", dict(x=t(2, 8), weight=t(8), residual=t(2, 8)), {}),
    ("norm_forward", dict(x=t(2, 8), weight=t(8), residual=t(2, 8)), dict(save=True)),
    ("norm_i8", dict(x=t(2, 8), weight=t(8), residual=t(2, 8)), {}),
    ("norm_backward", dict(dy=t(2, 8), total=t(2, 8), weight=t(8), rstd=t(2, dtype=F), dtotal=t(2, 8)), {}),
    ("balance_forward", dict(logits=t(2, 8, dtype=F)), dict(ids=torch.zeros(2, 2, dtype=I32))),
    ("balance_forward", dict(logits=t(2, 8, dtype=F)), dict(ids=torch.zeros(2, 2, dtype=I32), save=True)),
    ("balance_backward", dict(dlosses=t(2, dtype=F), logits=t(2, 8, dtype=F)),
     dict(counts=torch.zeros(9, dtype=I32), k=2)),
    ("lora_forward", dict({n: LORA[n] for n in ("x", "a", "b", "scale")}, base=t(2, 4)), dict(ids=LORA["ids"])),
    ("lora_forward", dict({n: LORA[n] for n in ("x", "a", "b", "scale")}, base=t(2, 4)), dict(ids=LORA["ids"], save=True)),
    ("lora_backward", dict({n: LORA[n] for n in ("x", "a", "b", "scale")}, dy=t(2, 4), t=t(2, 2, dtype=F), dx_base=t(2, 8)),
     dict(ids=LORA["ids"])),
]


@pytest.mark.parametrize("i,name", [(i, n) for i, c in enumerate(CALLS) for n in c[1]])
def test_operands_with_a_tangent_are_refused(i, name):
    fn, ops, rest = CALLS[i]
    call = getattr(B, fn)
    with fwd.dual_level():
        v = fwd.make_dual(ops[name], torch.ones_like(ops[name]))
        for ctx in (torch.enable_grad(), torch.no_grad()):
            with ctx, pytest.raises(B.MoeError, match=f"{fn}: {name} carries a tangent"):
                call(**{**ops, name: v}, **rest)
        # without one the call goes on (here to the check of the device)
        with pytest.raises(B.MoeError, match="needs device memory"):
            call(**ops, **rest)
        with pytest.raises(B.MoeError, match="needs device memory"):
            call(**{**ops, name: fwd.unpack_dual(v).primal}, **rest)
    with pytest.raises(B.MoeError, match="needs device memory"):
        call(**ops, **rest)
