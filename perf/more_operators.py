"""What stands around a layer's feed-forward block: cases, plain forms and definitions.

  norm        residual addition and root-mean-square norm in 16 bits
  norm_i8     the same with the result in 8 bits, a scale a row
  norm_train  the norm with its backward pass: y, total, then dx and dw from dy and dtotal
  balance     per-expert counts, balance loss and z loss of a router, then the logits' gradient
  lora        low-rank adapters, one a row, beside a shared projection's result
  lora_train  the same with its backward pass: y, then dx, da and db from dy

Definitions:
  norm: total = x + residual (in 32 bits, rounded to the type of the result),
    y = total w / sqrt(mean(total^2) + eps). In 8 bits: v = fp32(total w), s0 = fp32(max|v| / 127),
    q = round-half-even(v / s0), and the values q fp32(s0 / sqrt(...)); a row of zeros is zero.
  balance: over the n rows that the mask keeps, f_e = counts_e / (n k), P_e = mean softmax(l)_e,
    loss = E sum f_e P_e and mean(logsumexp(l)^2); the counts are constants to the gradient.
  lora: y_r = base_r + scale_i b_i (a_i x_r) with i = ids_r; rows with no adapter (-1) keep base_r.

`run` takes the plain form in elementary torch operations, or with `own` the calls of this package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one decode row: the experts' fp32 result joins the residual stream (latency)
        dict(name="norm-1row-bf16", kind="norm", rows=1, hidden=2048, dtype="bf16", x="fp32", residual=True),
        # a long prompt at the widest hidden size that a layer may have
        dict(name="norm-8192rows-fp16", kind="norm", rows=8192, hidden=4096, dtype="fp16", x="fp16", residual=True),
        # the widest decode step in front of an 8-bit product
        dict(name="norm_i8-16rows-bf16", kind="norm_i8", rows=16, hidden=2048, dtype="bf16", x="bf16", residual=True),
        # a ragged chunk of rows that are not 16-byte aligned, the first norm of a stack (no residual yet)
        dict(name="norm_i8-2077rows-odd-fp16", kind="norm_i8", rows=2077, hidden=1283, dtype="fp16", x="fp16",
             residual=False),
        # a short training batch at an odd size
        dict(name="norm_train-517rows-odd-fp16", kind="norm_train", rows=517, hidden=1283, dtype="fp16", x="fp16",
             residual=False),
        # a full training batch: gradients come from the block and along the residual stream
        dict(name="norm_train-8192rows-bf16", kind="norm_train", rows=8192, hidden=4096, dtype="bf16", x="bf16",
             residual=True),
        # a short training batch of a small router (latency)
        dict(name="balance-64rows-64experts", kind="balance", rows=64, experts=64, k=4, dtype="fp32", mask=False,
             beside=False),
        # a full training batch of the 256-expert router: its logits stand beside the shared gate's in one
        # buffer (odd rows), and padded rows do not count
        dict(name="balance-65536rows-256experts", kind="balance", rows=65536, experts=256, k=8, dtype="fp32",
             mask=True, beside=True),
        # a decode step: every row a request, every request an adapter of its own
        dict(name="lora-16rows-bf16", kind="lora", rows=16, n_in=2048, n_out=2048, rank=16, adapters=32, requests=16,
             dtype="bf16"),
        # prompts of many requests through a square projection
        dict(name="lora-4096rows-bf16", kind="lora", rows=4096, n_in=4096, n_out=4096, rank=64, adapters=8,
             requests=24, dtype="bf16"),
        # a training step at sizes that no tile divides, rows not 16-byte aligned
        dict(name="lora_train-777rows-odd-fp16", kind="lora_train", rows=777, n_in=1283, n_out=769, rank=20,
             adapters=3, requests=5, dtype="fp16"),
        # a full training batch of many adapters (the largest)
        dict(name="lora_train-8192rows-bf16", kind="lora_train", rows=8192, n_in=4096, n_out=4096, rank=64,
             adapters=16, requests=32, dtype="bf16"),
    ]


def _log(rng, lo, hi, even=True):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if even and rng.random() < 0.5:          # half the sizes as models have them, half as they fall
        step = 64 if v >= 256 else 8
        v = v // step * step
    return min(max(v, lo), hi)


def draw(rng):
    kind = rng.choice(["norm", "norm_i8", "norm_train", "balance", "lora", "lora_train"])
    if kind == "balance":
        experts = _log(rng, 8, 256)
        return dict(kind=kind, rows=_log(rng, 1, 65536), experts=experts, k=rng.randint(1, 8),
                    dtype=rng.choice(["fp32", "fp32", "bf16"]), mask=rng.random() < 0.5, beside=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "fp16"])
    if kind in ("lora", "lora_train"):
        rows = _log(rng, 1, 4096)
        requests = rows if rng.random() < 0.3 else _log(rng, 1, rows, even=False)
        return dict(kind=kind, rows=rows, n_in=_log(rng, 64, 4096), n_out=_log(rng, 64, 4096), rank=_log(rng, 4, 64),
                    adapters=_log(rng, 1, 32, even=False), requests=requests, dtype=dtype)
    residual = rng.random() < 0.7
    return dict(kind=kind, rows=_log(rng, 1, 8192), hidden=_log(rng, 64, 4096), dtype=dtype,
                x="fp32" if residual and rng.random() < 0.3 else dtype, residual=residual)


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * std


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) % (1 << 63))
    dt = DTYPES[case["dtype"]]
    R = case["rows"]
    st = dict(case=case)
    if case["kind"] == "balance":
        E = case["experts"]
        wide = _normal(gen, R, E + 1 if case["beside"] else E, std=1.5)
        # some experts are liked more than others
        wide[:, :E] += _normal(gen, E, std=0.7)
        wide = wide.to(dt)
        st["logits"] = wide[:, :E]
        st["ids"] = st["logits"].float().topk(case["k"], dim=1).indices.to(torch.int32)
        st["mask"] = torch.rand(R, generator=gen, device="cuda") < 0.9 if case["mask"] else None
        # the losses' weights in the training loss
        st["dloss"] = torch.tensor([1e-2, 1e-3], device="cuda") * (0.5 + torch.rand(2, generator=gen, device="cuda"))
        return st
    if case["kind"] in ("lora", "lora_train"):
        n, r, ni, no = case["adapters"], case["rank"], case["n_in"], case["n_out"]
        st["x"] = _normal(gen, R, ni).to(dt)
        st["a"] = _normal(gen, n, r, ni, std=1.0 / math.sqrt(ni)).to(dt)
        st["b"] = _normal(gen, n, no, r, std=0.3 / math.sqrt(r)).to(dt)
        st["scale"] = 0.5 + torch.rand(n, generator=gen, device="cuda")
        st["base"] = _normal(gen, R, no).to(dt)
        # requests of ragged lengths, their rows together; every eighth has no adapter
        S = case["requests"]
        cuts = torch.randperm(R - 1, generator=gen, device="cuda")[:S - 1] + 1
        first = torch.zeros(R, dtype=torch.int64, device="cuda")
        first[cuts] = 1
        request = torch.cumsum(first, 0)
        adapter = torch.randperm(n, generator=gen, device="cuda")[(request - request // 8) % n]
        st["ids"] = torch.where(request % 8 == 7, -1, adapter).to(torch.int32)
        if case["kind"] == "lora_train":
            st["dy"] = _normal(gen, R, no).to(dt)
            st["dx_base"] = _normal(gen, R, ni).to(dt)
        return st
    H = case["hidden"]
    x = _normal(gen, R, H)
    # a few strong channels, as hidden states have them
    strong = torch.rand(H, generator=gen, device="cuda") < 0.01
    x = torch.where(strong, x * 8.0, x)
    st["x"] = x.to(DTYPES[case["x"]])
    st["residual"] = (_normal(gen, R, H) * torch.where(strong, 8.0, 1.0)).to(dt) if case["residual"] else None
    st["w"] = (1.0 + _normal(gen, H, std=0.2)).to(dt)
    if case["kind"] == "norm_train":
        st["dy"] = _normal(gen, R, H).to(dt)
        st["dtotal"] = _normal(gen, R, H).to(dt) if case["residual"] else None
    return st


# ------------------------------------------------------------------ one pass
def _plain_norm(st):
    c, dt = st["case"], DTYPES[st["case"]["dtype"]]
    x, w = st["x"].float(), st["w"].float()
    total = None
    if st["residual"] is not None:
        total = (x + st["residual"].float()).to(dt)
        x = total.float()
    rs = 1.0 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS)
    if c["kind"] == "norm":
        return dict(y=(x * rs * w).to(dt), total=total)
    if c["kind"] == "norm_i8":
        v = x * w
        # 64 bits for the quotients: values next to a rounding border
        s0 = (v.abs().amax(dim=1, keepdim=True).double() / 127.0).float()
        q = torch.round(v.double() / s0.double()).clamp(-127, 127)
        q = torch.where(s0 > 0, q, torch.zeros_like(q)).float()
        return dict(values=q * (s0 * rs), total=total)
    dy = st["dy"].float()
    g = dy * w
    dx = rs * (g - x * rs * rs * (g * x).mean(dim=1, keepdim=True))
    if st["dtotal"] is not None:
        dx = dx + st["dtotal"].float()
    return dict(y=(x * rs * w).to(dt), total=total, dx=dx.to(dt), dw=(dy * x * rs).sum(dim=0).to(dt))


def _plain_balance(st):
    c, ids = st["case"], st["ids"].long()
    E, k = c["experts"], c["k"]
    l = st["logits"].float()
    keep = torch.ones(c["rows"], device=l.device) if st["mask"] is None else st["mask"].float()
    top = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - top)
    z = e.sum(dim=1, keepdim=True)
    p = e / z
    lse = (top + torch.log(z)).squeeze(1)
    counts = torch.zeros(E, dtype=torch.int32, device=l.device)
    counts.index_add_(0, ids.reshape(-1), keep.int().repeat_interleave(k))
    n = keep.sum().clamp(min=1.0)
    f = counts.float() / (n * k)
    losses = torch.stack([E * (f * (p * keep[:, None]).sum(dim=0)).sum() / n, (lse * lse * keep).sum() / n])
    gl, gz = st["dloss"][0], st["dloss"][1]
    d = p * (gl * E * (f - (p * f).sum(dim=1, keepdim=True)) + 2.0 * gz * lse[:, None]) * (keep / n)[:, None]
    return dict(losses=losses, counts=counts, dlogits=d.to(st["logits"].dtype))


def _plain_lora(st):
    c, ids = st["case"], st["ids"]
    dt = st["x"].dtype
    x, base, scale = st["x"].float(), st["base"].float(), st["scale"]
    R, n, r = c["rows"], c["adapters"], c["rank"]
    if c["kind"] == "lora" and R < n:
        # fewer rows than adapters: each row's own
        i = ids.long().clamp(min=0)
        t = (st["a"][i].float() * x[:, None, :]).sum(dim=2)
        d = (st["b"][i].float() * t[:, None, :]).sum(dim=2) * scale[i][:, None]
        return (base + torch.where(ids[:, None] >= 0, d, torch.zeros_like(d))).to(dt)
    # all adapters as one product, a row's own ones kept
    mine = (ids[:, None] == torch.arange(n, device=ids.device, dtype=ids.dtype)).unsqueeze(2)
    a = st["a"].float().reshape(n * r, -1)
    b = st["b"].float().transpose(1, 2).reshape(n * r, -1)
    t = (x @ a.t()).reshape(R, n, r)
    t = (torch.where(mine, t, torch.zeros_like(t)) * scale[:, None]).reshape(R, n * r)
    y = (base + t @ b).to(dt)
    if c["kind"] == "lora":
        return y
    dy = st["dy"].float()
    dt_ = (dy @ b.t()).reshape(R, n, r)
    dt_ = (torch.where(mine, dt_, torch.zeros_like(dt_)) * scale[:, None]).reshape(R, n * r)
    dx = (st["dx_base"].float() + dt_ @ a).to(dt)
    da = (dt_.t() @ x).reshape(n, r, -1).to(dt)
    db = (t.t() @ dy).reshape(n, r, -1).transpose(1, 2).to(dt).contiguous()
    return dict(y=y, dx=dx, da=da, db=db)


def _own(st):
    import quantized_routed_expert_fp32_amd as qr
    c = st["case"]
    if c["kind"] == "norm":
        y, total, _ = qr.norm_forward(st["x"], st["w"], residual=st["residual"], eps=EPS)
        return dict(y=y, total=total)
    if c["kind"] == "norm_i8":
        q, scale, total, _ = qr.norm_i8(st["x"], st["w"], residual=st["residual"], eps=EPS)
        return dict(values=q * scale[:, None], total=total)
    if c["kind"] == "norm_train":
        y, total, rstd = qr.norm_forward(st["x"], st["w"], residual=st["residual"], eps=EPS, save=True)
        dx, dw = qr.norm_backward(st["dy"], st["x"] if total is None else total, st["w"], rstd, dtotal=st["dtotal"])
        return dict(y=y, total=total, dx=dx, dw=dw)
    if c["kind"] == "balance":
        losses, counts = qr.balance_forward(st["logits"], st["ids"], mask=st["mask"], save=True)
        d = qr.balance_backward(st["dloss"], st["logits"], counts, c["k"], mask=st["mask"])
        return dict(losses=losses, counts=counts[:-1], dlogits=d)
    if c["kind"] == "lora":
        return qr.lora_forward(st["x"], st["a"], st["b"], st["ids"], st["scale"], base=st["base"])
    y, t = qr.lora_forward(st["x"], st["a"], st["b"], st["ids"], st["scale"], base=st["base"], save=True)
    dx, da, db = qr.lora_backward(st["dy"], st["x"], st["a"], st["b"], st["ids"], st["scale"], t,
                                  dx_base=st["dx_base"])
    return dict(y=y, dx=dx, da=da, db=db)


def run(state):
    if own:
        return _own(state)
    if state["case"]["kind"] == "balance":
        return _plain_balance(state)
    if state["case"]["kind"] in ("lora", "lora_train"):
        return _plain_lora(state)
    return _plain_norm(state)


def work(case):
    R = case["rows"]
    if case["kind"] == "balance":
        E, k = case["experts"], case["k"]
        size = 4 if case["dtype"] == "fp32" else 2
        # the logits again for their gradient, which needs every row's counts
        return dict(bytes=R * (3 * size * E + 4 * k + (1 if case["mask"] else 0)) + 4 * E + 8, flops=12 * R * E)
    if case["kind"] in ("lora", "lora_train"):
        r, ni, no, S = case["rank"], case["n_in"], case["n_out"], case["requests"]
        used = min(case["adapters"], S - S // 8)
        first = 2 * (R * ni + 2 * R * no + used * r * (ni + no)) + 4 * R
        if case["kind"] == "lora":
            return dict(bytes=first, flops=2 * R * r * (ni + no))
        return dict(bytes=first + 2 * (R * no + 2 * R * ni + case["adapters"] * r * (ni + no)),
                    flops=6 * R * r * (ni + no))
    H, xs = case["hidden"], 4 if case["x"] == "fp32" else 2
    n = R * H
    b = xs * n + 2 * H + (4 * n if case["residual"] else 0)
    if case["kind"] == "norm":
        return dict(bytes=b + 2 * n, flops=4 * n)
    if case["kind"] == "norm_i8":
        return dict(bytes=b + n + 4 * R, flops=5 * n)
    # the norm's own input is read once and stays at hand; dy, dtotal and the gradients beside it
    return dict(bytes=b + 2 * n + 4 * n + (2 * n if case["residual"] else 0) + 2 * H, flops=14 * n)


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_norm(st):
    c = st["case"]
    f64 = torch.float64
    s = total = None
    if st["residual"] is None:
        s = st["x"].to(f64)
    else:
        total = st["x"].to(f64) + st["residual"].to(f64)
        # the rounding of the total is part of the definition
        s = torch.add(st["x"].to(torch.float32), st["residual"].to(torch.float32)).to(DTYPES[c["dtype"]]).to(f64)
    w = st["w"].to(f64)
    H = c["hidden"]
    root = torch.sqrt(torch.square(s).sum(1) / H + EPS).unsqueeze(1)
    if c["kind"] == "norm_i8":
        v = torch.mul(s, w).to(torch.float32).to(f64)
        step = (torch.linalg.vector_norm(v, ord=math.inf, dim=1, keepdim=True) / 127).to(torch.float32).to(f64)
        z = torch.where(step > 0, torch.round(v / torch.where(step > 0, step, 1.0)), 0.0)
        return dict(values=torch.clamp(z, -127.0, 127.0) * step / root, total=total)
    n = s / root
    out = dict(y=n * w, total=total)
    if c["kind"] == "norm_train":
        e = st["dy"].to(f64)
        ew = e * w
        dx = (ew - n * ((ew * n).sum(1) / H).unsqueeze(1)) / root
        out.update(dx=dx if st["dtotal"] is None else dx + st["dtotal"].to(f64), dw=(e * n).sum(0))
    return out


def _exact_balance(st):
    c = st["case"]
    E, k, R = c["experts"], c["k"], c["rows"]
    kept = torch.arange(R, device="cuda") if st["mask"] is None else torch.nonzero(st["mask"]).flatten()
    l = st["logits"].double()[kept]
    n = max(1, kept.numel())
    counts = torch.bincount(st["ids"].long()[kept].flatten(), minlength=E)
    f = counts.double() / (n * k)
    lse = torch.logsumexp(l, 1)
    p = torch.softmax(l, 1)
    losses = torch.stack([E * torch.dot(f, p.sum(0)) / n, torch.dot(lse, lse) / n])
    g = st["dloss"].double()
    inner = f.unsqueeze(0) - torch.mv(p, f).unsqueeze(1)
    d = torch.zeros(R, E, dtype=torch.float64, device="cuda")
    d[kept] = p / n * (g[0] * E * inner + 2 * g[1] * lse.unsqueeze(1))
    return dict(losses=losses, counts=counts.to(torch.int32), dlogits=d)


def _exact_lora(st):
    c = st["case"]
    y, x = st["base"].double(), st["x"].double()
    train = c["kind"] == "lora_train"
    a, b = st["a"].double(), st["b"].double()
    if train:
        dy, dx, da, db = st["dy"].double(), st["dx_base"].double(), torch.zeros_like(a), torch.zeros_like(b)
    for i in range(c["adapters"]):
        rows = torch.nonzero(st["ids"] == i).flatten()
        if not rows.numel():
            continue
        s = float(st["scale"][i])
        low = torch.matmul(x[rows], a[i].t().contiguous())
        y[rows] += s * torch.matmul(low, b[i].t().contiguous())
        if train:
            back = s * torch.matmul(dy[rows], b[i])
            dx[rows] += torch.matmul(back, a[i])
            da[i] = torch.matmul(back.t().contiguous(), x[rows])
            db[i] = s * torch.matmul(dy[rows].t().contiguous(), low)
    return dict(y=y, dx=dx, da=da, db=db) if train else y


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "balance":
        return _exact_balance(st)
    if case["kind"] in ("lora", "lora_train"):
        return _exact_lora(st)
    return _exact_norm(st)
