"""The operators around the feed-forward block as a layer uses them, one behind the
other, eager and captured."""
import pytest
import torch

import block_common as K
from gpu_common import binding, log

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rnd(g, *shape, std=1.0, dt=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)


@pytest.mark.parametrize("R", [1, 16, 300])
def test_serving(R):
    """Experts' fp32 result and residual through the norm into 8 bits, an 8-bit product, adapters beside it."""
    log(f"case together serving {R}")
    B = binding()
    g = torch.Generator(device="cuda")
    g.manual_seed(R)
    H, N, n = 512, 264, 5
    x, res, w = rnd(g, R, H), rnd(g, R, H, dt=BF), (1 + rnd(g, H, std=0.2)).to(BF)
    wq, sw = B.quant_rows(rnd(g, N, H, std=H ** -0.5))
    a, b = rnd(g, n, 8, H, std=H ** -0.5, dt=BF), rnd(g, n, N, 8, std=0.3, dt=BF)
    ids = torch.randint(-1, n, (R,), generator=g, device="cuda").to(torch.int32)
    scale = 0.5 + torch.rand(n, generator=g, device="cuda")

    def layer():
        q, s, total, y = B.norm_i8(x, w, residual=res, want_y=True)
        z = B.linear_i8(q, wq, sw, x_scale=s, out_dtype=BF)
        return q, s, total, y, z, B.lora_forward(y, a, b, ids, scale, base=z)

    q, s, total, y, z, out = layer()
    want = K.total_of(x, res, BF)
    assert torch.equal(total, want) and torch.equal(q.cpu(), K.norm_codes(want, w)[0])
    K.close(y, *K.norm(want, w, 1e-6, BF)[:2], "y")
    v = (q.double() @ wq.double().t()) * s.double().unsqueeze(1) * sw.double()
    K.close(z, v, K.rounded(v, 4 * K.U * v.abs(), BF), "z")
    K.close(out, *K.lora(y, a, b, ids, scale, z)[1], "out")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    for i in range(3):
        x.copy_(rnd(g, R, H))
        ids.copy_(torch.randint(-1, n, (R,), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, t) for p, t in zip(got, layer())), i


@pytest.mark.parametrize("R", [20, 400])
def test_training_step(R):
    """Norm, adapters beside a gated block's input, the block and a router's balance, and all
    gradients back to the stream, against 64-bit formulas on the values that the forward calls rounded."""
    log(f"case together training {R}")
    B = binding()
    g = torch.Generator(device="cuda")
    g.manual_seed(R)
    H, I, E, k, n = 128, 96, 16, 2, 3
    x, res, w = rnd(g, R, H, dt=BF), rnd(g, R, H, dt=BF), (1 + rnd(g, H, std=0.2)).to(BF)
    wg, wu = rnd(g, I, H, std=H ** -0.5, dt=BF), rnd(g, I, H, std=H ** -0.5, dt=BF)
    a, b = rnd(g, n, 4, H, std=H ** -0.5, dt=BF), rnd(g, n, H, 4, std=0.3, dt=BF)
    ids = torch.randint(-1, n, (R,), generator=g, device="cuda").to(torch.int32)
    scale = torch.ones(n, device="cuda")
    logits = rnd(g, R, E)
    picks = logits.topk(k, dim=1).indices.to(torch.int32)
    dh, dlosses = rnd(g, R, I, dt=BF), torch.tensor([0.01, 0.001], device="cuda")

    def step():
        y, total, rstd = B.norm_forward(x, w, residual=res, save=True)
        z, t = B.lora_forward(y, a, b, ids, scale, base=y, save=True)
        h, gu = B.glu_forward(z, wg, wu, save=True)
        losses, counts = B.balance_forward(logits, picks, save=True)
        dz, dwg, dwu = B.glu_backward(dh, z, wg, wu, gu)
        dy, da, db = B.lora_backward(dz, y, a, b, ids, scale, t, dx_base=dz)
        dx, dw = B.norm_backward(dy, total, w, rstd, dtotal=dy)
        dl = B.balance_backward(dlosses, logits, counts, k)
        return y, total, rstd, z, t, h, losses, counts, dz, dy, da, db, dx, dw, dl, dwg, dwu

    y, total, rstd, z, t, h, losses, counts, dz, dy, da, db, dx, dw, dl, dwg, dwu = eager = step()
    K.close(z, *K.lora(y, a, b, ids, scale, y)[1], "z")
    for name, v, want in zip(("dy", "da", "db"), (dy, da, db), K.lora_grads(dz, y, a, b, ids, scale, t, dz)):
        K.close(v, *want, name)
    for name, v, want in zip(("dx", "dw"), (dx, dw), K.norm_grads(dy, total, w, rstd, dy, BF)):
        K.close(v, *want, name)
    wl, wc, wd = K.balance(logits, picks, None, dlosses)
    K.close(losses, *wl, "losses")
    assert torch.equal(counts, wc)
    K.close(dl, *wd, "dlogits")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        x.copy_(rnd(g, R, H, dt=BF))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, step())), i
