"""GPU parity of the balance losses, the counts and the logits' gradient against
their plain 64-bit forms (tests/block_common.py derives the bounds)."""
import pytest
import torch

import block_common as K
from gpu_common import binding, log

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
IDS = {BF: "bf16", FP: "fp16", F32: "fp32"}


def inputs(seed, R, E, k, dt, masked=None, std=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    l = (torch.randn(R, E, generator=g, device="cuda") * std).to(dt)
    ids = l.float().topk(k, dim=1).indices.to(torch.int32)
    mask = None if masked is None else torch.rand(R, generator=g, device="cuda") >= masked
    d = torch.tensor([0.3, -0.7], device="cuda")
    return l, ids, mask, d


def check(B, l, ids, mask, d):
    losses, counts = B.balance_forward(l, ids, mask=mask)
    dl = B.balance_backward(d, l, counts, ids.shape[1], mask=mask)
    (wl, bl), wc, (wd, bd) = K.balance(l, ids, mask, d)
    assert torch.equal(counts, wc)
    K.close(losses, wl, bl, "losses")
    assert dl.dtype == l.dtype and dl.is_contiguous()
    K.close(dl, wd, bd, "dlogits")
    # again: the same bits
    l2, c2 = B.balance_forward(l, ids, mask=mask)
    assert torch.equal(l2, losses) and torch.equal(B.balance_backward(d, l, c2, ids.shape[1], mask=mask), dl)
    return losses, counts, dl


# each width of a row's lanes, ragged ends, one workgroup and several
SIZES = [(1, 1, 1), (1, 8, 1), (3, 5, 2), (64, 64, 4), (17, 63, 8), (256, 65, 3), (257, 128, 8), (300, 129, 2),
         (1000, 256, 8), (513, 255, 1), (40, 257, 8), (700, 511, 6), (300, 1000, 8), (9, 1024, 64), (8200, 64, 2),
         (20000, 256, 8), (9000, 40, 40)]


@pytest.mark.parametrize("dt", [F32, BF, FP], ids=IDS.get)
@pytest.mark.parametrize("R,E,k", SIZES)
def test_sizes(R, E, k, dt):
    log(f"case balance {R} {E} {k} {dt}")
    B = binding()
    for masked in (None, 0.3):
        check(B, *inputs(R + E, R, E, k, dt, masked))


@pytest.mark.parametrize("E", [7, 64, 256, 300])
def test_rows_beside_the_shared_gate(E):
    """Logits in rows of E + 1, and a gradient written into such rows: the last column stays."""
    log(f"case balance strides {E}")
    B = binding()
    l, ids, mask, d = inputs(E, 333, E, 4, F32, 0.2)
    wide = torch.full((333, E + 1), float("nan"), device="cuda")
    wide[:, :E] = l
    losses, counts, dl = check(B, wide[:, :E], ids, mask, d)
    ref = B.balance_forward(l, ids, mask=mask)
    assert torch.equal(ref[0], losses) and torch.equal(ref[1], counts)
    out = torch.full((333, E + 1), 7.0, device="cuda")
    B.balance_backward(d, wide[:, :E], counts, 4, mask=mask, dlogits=out[:, :E])
    assert torch.equal(out[:, :E], dl) and (out[:, E] == 7.0).all()


def test_rows_that_do_not_count():
    """Whatever stands in masked rows; no row at all; picks outside the experts."""
    B = binding()
    for R, E in ((100, 64), (600, 256)):
        log(f"case balance masks {R} {E}")
        l, ids, mask, d = inputs(1, R, E, 4, F32, 0.5)
        want = check(B, l, ids, mask, d)
        l2, ids2 = l.clone(), ids.clone()
        l2[~mask] = float("nan")
        ids2[~mask] = 1 << 30
        got = check(B, l2, ids2, mask, d)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and (got[2][~mask] == 0).all()
        none = torch.zeros_like(mask)
        losses, counts, dl = check(B, l2 * 0 + float("inf"), ids2, none, d)
        assert (losses == 0).all() and (counts == 0).all() and (dl == 0).all()
        ids[::3, 1] = -1
        ids[1::3, 0] = E
        _, counts, _ = check(B, l, ids, None, d)
        assert counts[:E].sum() == ids.numel() - len(ids[::3]) - len(ids[1::3]) and counts[E] == R


def test_experts_taken_out_and_far_logits():
    B = binding()
    for R, E in ((50, 60), (400, 256)):
        log(f"case balance extremes {R} {E}")
        for dt in (F32, BF):
            l, ids, _, d = inputs(2, R, E, 3, dt)
            l[:, 5] = -float("inf")
            l[:, 6] = torch.finfo(dt).min
            l[7] = -float("inf")
            l[7, 3] = 2.0                       # one expert left
            l[8] += 1000.0
            l[9] *= 40.0
            l[10] = 0.0
            ids = l.float().topk(3, dim=1).indices.to(torch.int32)
            _, _, dl = check(B, l, ids, None, d)
            out = l.float() <= torch.finfo(dt).min            # (row 10 has them in again)
            assert out.sum() > 2 * (R - 2) and (dl[out] == 0).all()
        # rows without a softmax: the losses say so, the other rows keep their gradient
        bad = l.clone()
        bad[0] = -float("inf")
        losses, counts = B.balance_forward(bad, ids)
        assert losses.isnan().all() and torch.equal(counts, B.balance_forward(l, ids)[1])
        dl2 = B.balance_backward(d, bad, counts, 3)
        assert dl2[0].isnan().all() and torch.equal(dl2[1:], dl[1:])
        for v in (float("nan"), float("inf")):
            bad[0] = l[0]
            bad[0, E - 1] = v
            assert B.balance_forward(bad, ids)[0].isnan().all()


def test_an_even_load_and_differences():
    B = binding()
    log("case balance differences")
    R, E, k = 64, 8, 2
    ids = (torch.arange(R * k, device="cuda") % E).reshape(R, k).to(torch.int32)
    losses, _ = B.balance_forward(torch.zeros(R, E, device="cuda"), ids)
    assert abs(losses[0].item() - 1) < 1e-6 and abs(losses[1].item() - torch.tensor(8.0).log().item() ** 2) < 1e-5
    l, ids, mask, d = inputs(3, 12, 6, 2, F32, 0.3)
    _, counts = B.balance_forward(l, ids, mask=mask)
    dl = B.balance_backward(d, l, counts, 2, mask=mask)
    n, f = int(counts[6]), counts[:6].double() / (int(counts[6]) * 2)

    def loss(v):
        v = v[mask]
        lse = torch.logsumexp(v, 1)
        return d[0].double() * 6 * (f * torch.softmax(v, 1).sum(0)).sum() / n + d[1].double() * (lse * lse).sum() / n

    h, want = 1e-6, torch.zeros(12, 6, dtype=torch.float64, device="cuda")
    for i in range(12):
        for j in range(6):
            e = torch.zeros_like(want)
            e[i, j] = h
            want[i, j] = (loss(l.double() + e) - loss(l.double() - e)) / (2 * h)
    _, _, (_, bd) = K.balance(l, ids, mask, d)
    K.close(dl, want, bd + 1e-8, "difference")


def test_with_the_router():
    """ids and logits as route gives them (rows beside the shared gate's logit)."""
    import synth
    from synth import to_abi
    B = binding()
    spec = synth.make_tiny_config(synth.CONFIGS[0], cfg_id=901, hidden=512, n_experts=64, top_k=4, inter=256,
                                  shared_inter=256)
    layer = B.pack_layer(B.layer_desc(*to_abi.desc_args(spec)), to_abi.tensors(synth.make_layer(spec, 0)))
    R = 24
    x = torch.from_numpy(synth.make_x(spec, 0, R, rep=1).view("int16")).cuda()
    log("case balance router")
    logits = torch.empty(R, 65, device="cuda")
    ids, _, _ = B.route(layer, x, taps={"logits": logits})
    d = torch.tensor([0.01, 0.001], device="cuda")
    check(B, logits[:, :64], ids, None, d)


def test_streams_and_graphs():
    B = binding()
    log("case balance graphs")
    for R in (200, 3000):
        l, ids, mask, d = inputs(R, R, 256, 8, F32, 0.2)

        def call(stream=None):
            losses, counts = B.balance_forward(l, ids, mask=mask, stream=stream)
            return losses, counts, B.balance_backward(d, l, counts, 8, mask=mask, stream=stream)

        want = call()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = call(s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        for i in range(4):
            l.copy_(inputs(i + 10, R, 256, 8, F32)[0])
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, call())), i
