"""The dense feed-forward operators beside the routed experts: cases, plain forms and definitions.

  glu    h = act(x Wg^T) * (x Wu^T) in 16 bits, from one row to long chunks
  train  the same with its backward pass: h, then dx, dWg and dWu from dh
  i8     y = x W^T (+ bias) with 8-bit weights (a scale a channel) and x quantised a token
  glu_i8 the gated block on 8-bit weights

The 8-bit quantisation of a row v: s = fp32(max|v| / 127), q = round-half-even(v / s) within
-127..127; a row of zeros has s = 0 and q = 0. `run` takes the plain form in elementary torch
operations, or with `own` the calls of this package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one decode row through a block of the experts' width (latency)
        dict(name="glu-1row-bf16", kind="glu", rows=1, hidden=2048, inter=512, dtype="bf16", act="silu"),
        # the widest decode step of the widest layer the library accepts
        dict(name="glu-16rows-fp16", kind="glu", rows=16, hidden=4096, inter=2048, dtype="fp16", act="gelu_tanh"),
        # a prompt chunk through the dense block of a model of this hidden size
        dict(name="glu-2048rows-bf16", kind="glu", rows=2048, hidden=2048, inter=8192, dtype="bf16", act="silu"),
        # a training step of a shared expert on a short batch
        dict(name="train-512rows-bf16", kind="train", rows=512, hidden=2048, inter=512, dtype="bf16", act="silu"),
        # sizes no tile divides and rows that are not 16-byte aligned
        dict(name="train-777rows-odd-fp16", kind="train", rows=777, hidden=1283, inter=769, dtype="fp16",
             act="gelu_tanh"),
        # a training step of a dense block on a full batch (the largest)
        dict(name="train-8192rows-bf16", kind="train", rows=8192, hidden=4096, inter=8192, dtype="bf16", act="silu"),
        # one decode row through a square projection
        dict(name="i8-1row-bf16", kind="i8", rows=1, hidden=2048, out=2048, dtype="bf16", bias=False),
        # a ragged chunk, odd sizes and a bias
        dict(name="i8-333rows-odd-fp16", kind="i8", rows=333, hidden=1283, out=777, dtype="fp16", bias=True),
        # a long prompt through a wide projection
        dict(name="i8-8192rows-bf16", kind="i8", rows=8192, hidden=4096, out=8192, dtype="bf16", bias=False),
        # a window of decode rows
        dict(name="glu_i8-16rows-bf16", kind="glu_i8", rows=16, hidden=2048, inter=512, dtype="bf16", act="silu"),
        # a ragged chunk of the odd layer shape
        dict(name="glu_i8-517rows-fp16", kind="glu_i8", rows=517, hidden=1280, inter=768, dtype="fp16",
             act="gelu_tanh"),
        # a long prompt through the dense block
        dict(name="glu_i8-4096rows-bf16", kind="glu_i8", rows=4096, hidden=4096, inter=8192, dtype="bf16",
             act="silu"),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:          # half the sizes as models have them, half as they fall
        step = 64 if v >= 256 else 8
        v = v // step * step
    return min(max(v, lo), hi)


def draw(rng):
    kind = rng.choice(["glu", "train", "i8", "glu_i8"])
    c = dict(kind=kind, rows=_log(rng, 1, 4096), hidden=_log(rng, 64, 4096), dtype=rng.choice(["bf16", "fp16"]))
    if kind == "i8":
        c.update(out=_log(rng, 64, 8192), bias=rng.random() < 0.5)
    else:
        c.update(inter=_log(rng, 64, 8192), act=rng.choice(["silu", "gelu_tanh"]))
    return c


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _codes(gen, n, k):
    """8-bit weights as a channel-wise quantisation of normal weights leaves them, and their scales."""
    q = torch.clamp(torch.round(_normal(gen, n, k, std=32.0)), -127, 127).to(torch.int8)
    s = (0.5 + torch.rand(n, generator=gen, device="cuda")) / (32.0 * math.sqrt(k))
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) % (1 << 63))
    dt = DTYPES[case["dtype"]]
    M, H = case["rows"], case["hidden"]
    st = dict(case=case)
    x = _normal(gen, M, H)
    if case["kind"] in ("i8", "glu_i8"):
        # a few strong channels, as hidden states have them
        strong = torch.rand(H, generator=gen, device="cuda") < 0.01
        x = torch.where(strong, x * 8.0, x)
    st["x"] = x.to(dt)
    if case["kind"] == "i8":
        st["w"] = _codes(gen, case["out"], H)
        st["bias"] = _normal(gen, case["out"]) if case["bias"] else None
    elif case["kind"] == "glu_i8":
        st["gate"], st["up"] = _codes(gen, case["inter"], H), _codes(gen, case["inter"], H)
    else:
        I = case["inter"]
        st["wg"] = _normal(gen, I, H, std=1.0 / math.sqrt(H)).to(dt)
        st["wu"] = _normal(gen, I, H, std=1.0 / math.sqrt(H)).to(dt)
        if case["kind"] == "train":
            st["dh"] = _normal(gen, M, I).to(dt)
    return st


# ------------------------------------------------------------------ one pass
_C = math.sqrt(2.0 / math.pi)


def _act(g, act):
    """The activation and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    t = torch.tanh(_C * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * _C * (1.0 + 3 * 0.044715 * g * g)


def _plain_quant(x):
    amax = x.abs().amax(dim=1, keepdim=True).float()
    s = amax / 127.0
    # 64 bits for the quotient: values next to a rounding border
    q = torch.round(x.double() / s.double()).clamp(-127, 127)
    return torch.where(s > 0, q, torch.zeros_like(q)).float(), s


def _plain(st):
    c, x = st["case"], st["x"]
    dt = x.dtype
    if c["kind"] == "i8":
        q, s = _plain_quant(x)
        y = (q @ st["w"][0].float().t()) * s * st["w"][1]
        if st["bias"] is not None:
            y = y + st["bias"]
        return y.to(dt)
    if c["kind"] == "glu_i8":
        q, s = _plain_quant(x)
        g = (q @ st["gate"][0].float().t()) * s * st["gate"][1]
        u = (q @ st["up"][0].float().t()) * s * st["up"][1]
        return (_act(g, c["act"])[0] * u).to(dt)
    xf, wg, wu = x.float(), st["wg"].float(), st["wu"].float()
    g, u = xf @ wg.t(), xf @ wu.t()
    a, da = _act(g, c["act"])
    h = (a * u).to(dt)
    if c["kind"] == "glu":
        return h
    dh = st["dh"].float()
    dg, du = dh * u * da, dh * a
    return dict(h=h, dx=(dg @ wg + du @ wu).to(dt), dw_gate=(dg.t() @ xf).to(dt), dw_up=(du.t() @ xf).to(dt))


def _own(st):
    import quantized_routed_expert_fp32_amd as qr
    c, x = st["case"], st["x"]
    if c["kind"] == "i8":
        return qr.linear_i8(x, *st["w"], bias=st["bias"])
    if c["kind"] == "glu_i8":
        return qr.glu_i8(x, *st["gate"], *st["up"], act=c["act"])
    if c["kind"] == "glu":
        return qr.glu_forward(x, st["wg"], st["wu"], act=c["act"])
    h, gu = qr.glu_forward(x, st["wg"], st["wu"], act=c["act"], save=True)
    dx, dwg, dwu = qr.glu_backward(st["dh"], x, st["wg"], st["wu"], gu, act=c["act"])
    return dict(h=h, dx=dx, dw_gate=dwg, dw_up=dwu)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    M, H = case["rows"], case["hidden"]
    if case["kind"] == "i8":
        N = case["out"]
        return dict(bytes=2 * M * H + N * H + 4 * N * (2 if case["bias"] else 1) + 2 * M * N, flops=2 * M * N * H)
    I = case["inter"]
    if case["kind"] == "glu_i8":
        return dict(bytes=2 * M * H + 2 * I * H + 8 * I + 2 * M * I, flops=4 * M * H * I)
    if case["kind"] == "glu":
        return dict(bytes=2 * (M * H + 2 * I * H + M * I), flops=4 * M * H * I)
    return dict(bytes=2 * (2 * M * H + 4 * I * H + 2 * M * I), flops=12 * M * H * I)


# ------------------------------------------------------------------ the definition in 64 bits
def _phi(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    return z * torch.sigmoid(2.0 * _C * (z + 0.044715 * z ** 3))


def _dphi(z, act):
    # z * sigmoid(w(z)): sigmoid + z * sigmoid' * w'
    w, dw = (z, torch.ones_like(z)) if act == "silu" else (2.0 * _C * (z + 0.044715 * z ** 3),
                                                          2.0 * _C * (1.0 + 0.134145 * z ** 2))
    p = torch.sigmoid(w)
    return p + z * p * torch.sigmoid(-w) * dw


def _dequant_rows(x):
    """The values that x's 8-bit codes stand for, and the codes' scales (which are 32-bit numbers)."""
    top = torch.amax(torch.abs(x.to(torch.float32)), 1).cpu()
    s = (top / torch.tensor(127.0)).to(x.device).double().unsqueeze(1)
    z = x.double()
    return torch.where(s > 0, s * torch.clamp(torch.round(z / torch.where(s > 0, s, 1.0)), -127.0, 127.0), 0.0)


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind in ("i8", "glu_i8"):
        xv = _dequant_rows(st["x"])
        mat = lambda w: w[1].double().unsqueeze(1) * w[0].double()
        if kind == "i8":
            y = torch.matmul(xv, mat(st["w"]).t().contiguous())
            return y if st["bias"] is None else y + st["bias"].double()
        z = torch.matmul(xv, mat(st["gate"]).t().contiguous())
        return _phi(z, case["act"]) * torch.matmul(xv, mat(st["up"]).t().contiguous())
    x, wg, wu = st["x"].double(), st["wg"].double(), st["wu"].double()
    z, v = torch.matmul(x, wg.t().contiguous()), torch.matmul(x, wu.t().contiguous())
    h = _phi(z, case["act"]) * v
    if kind == "glu":
        return h
    e = st["dh"].double()
    dz, dv = e * v * _dphi(z, case["act"]), e * _phi(z, case["act"])
    dx = torch.matmul(dz, wg) + torch.matmul(dv, wu)
    return dict(h=h, dx=dx, dw_gate=torch.matmul(dz.t().contiguous(), x), dw_up=torch.matmul(dv.t().contiguous(), x))
