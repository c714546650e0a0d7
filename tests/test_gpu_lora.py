"""GPU parity of the low-rank adapters and their gradients against their plain
64-bit forms (tests/block_common.py derives the bounds)."""
import pytest
import torch

import block_common as K
from gpu_common import binding, log

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
IDS = {BF: "bf16", FP: "fp16"}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, std=1.0, dt=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)


def rows_of(kind, g, R, n):
    """Adapters of the rows: ragged runs, any order, one for all, none at all."""
    if kind == "none":
        return torch.full((R,), -1, device="cuda", dtype=torch.int32)
    if kind == "one":
        return torch.full((R,), n - 1, device="cuda", dtype=torch.int32)
    ids = torch.randint(-1, n, (R,), generator=g, device="cuda")
    if kind == "runs":
        start = torch.rand(R, generator=g, device="cuda") < 0.05
        ids = ids[torch.cumsum(start, 0)]
    return ids.to(torch.int32)


def problem(seed, R, K_, N, rank, n, dt, kind):
    g = gen(seed)
    return dict(x=rnd(g, R, K_, dt=dt), a=rnd(g, n, rank, K_, std=K_ ** -0.5, dt=dt),
                b=rnd(g, n, N, rank, std=rank ** -0.5, dt=dt), ids=rows_of(kind, g, R, n),
                scale=0.5 + torch.rand(n, generator=g, device="cuda")), g


def check(B, p, g, base=True, grads=True):
    x, b, dt = p["x"], p["b"], p["x"].dtype
    R, N = x.shape[0], b.shape[1]
    base = rnd(g, R, N, dt=dt) if base else None
    y, t = B.lora_forward(**p, base=base, save=True)
    (wt, bt), (wy, by) = K.lora(**p, base=base)
    K.close(t, wt, bt, "t")
    K.close(y, wy, by, "y")
    none = (p["ids"] < 0) | (p["ids"] >= b.shape[0])
    assert torch.equal(y[none], base[none] if base is not None else torch.zeros_like(y[none])) and (t[none] == 0).all()
    assert torch.equal(B.lora_forward(**p, base=base), y)
    if grads:
        dy, dxb = rnd(g, R, N, dt=dt), rnd(g, *x.shape, dt=dt)
        check_grads(B, p, dy, t, dxb)
        check_grads(B, p, dy, t, None)
    return y, t


def check_grads(B, p, dy, t, dxb):
    got = B.lora_backward(dy, **p, t=t, dx_base=dxb)
    for name, v, (want, bound) in zip(("dx", "da", "db"), got, K.lora_grads(dy, **p, t=t, dx_base=dxb)):
        K.close(v, want, bound, name)
    none = (p["ids"] < 0) | (p["ids"] >= p["b"].shape[0])
    assert torch.equal(got[0][none], dxb[none] if dxb is not None else torch.zeros_like(got[0][none]))
    # again, and one at a time: the same bits
    dx, n1, n2 = B.lora_backward(dy, **p, dx_base=dxb, need_dw=False)
    assert n1 is None and n2 is None and torch.equal(dx, got[0])
    n0, da, db = B.lora_backward(dy, **p, t=t, need_dx=False)
    assert n0 is None and torch.equal(da, got[1]) and torch.equal(db, got[2])
    return got


# rows x in x out, rank, adapters: one row, few rows, tile edges, odd sizes
SIZES = [(1, 64, 64, 8, 1), (1, 1, 1, 1, 1), (16, 2048, 2048, 16, 32), (2, 7, 3, 2, 2), (64, 1283, 77, 4, 3), (40, 100, 600, 33, 5),
         (65, 64, 64, 16, 2), (100, 130, 70, 17, 3), (128, 2048, 512, 32, 4), (200, 1283, 769, 20, 3), (70, 9, 1, 3, 2),
         (300, 520, 1030, 64, 2), (257, 264, 131, 65, 4), (130, 72, 4100, 100, 2), (77, 4104, 40, 256, 3),
         (1000, 200, 136, 8, 300), (4200, 136, 264, 24, 5), (5000, 520, 72, 129, 3)]


@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
@pytest.mark.parametrize("kind", ["runs", "any"])
@pytest.mark.parametrize("R,K_,N,rank,n", SIZES)
def test_sizes(R, K_, N, rank, n, dt, kind):
    log(f"case lora {R} {K_} {N} {rank} {n} {dt} {kind}")
    B = binding()
    p, g = problem(R + K_ + rank, R, K_, N, rank, n, dt, kind)
    check(B, p, g)
    check(B, p, g, base=False, grads=False)


@pytest.mark.parametrize("rank", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 31, 32, 63, 64, 128, 255])
def test_ranks(rank):
    log(f"case lora rank {rank}")
    B = binding()
    for R in (3, 90):
        p, g = problem(rank, R, 130, 134, rank, 4, BF if rank % 2 else FP, "any")
        check(B, p, g)


@pytest.mark.parametrize("kind", ["none", "one"])
@pytest.mark.parametrize("R", [1, 5, 64, 70, 1500, 8192])
def test_one_adapter_or_none(R, kind):
    """All rows on the last of three adapters (several segments of gradients for the
    long ones, zeros for the others), or on none."""
    log(f"case lora {kind} {R}")
    B = binding()
    p, g = problem(R, R, 200, 136, 16, 3, BF, kind)
    check(B, p, g)


@pytest.mark.parametrize("R,n", [(8193, 3), (20000, 40), (30000, 1024), (16384, 1)])
def test_many_rows(R, n):
    """More rows than one sorting workgroup takes."""
    log(f"case lora rows {R} {n}")
    B = binding()
    p, g = problem(R, R, 72, 40, 8, n, FP if n == 40 else BF, "any")
    check(B, p, g)
    p["ids"] = rows_of("one", g, R, n)
    check(B, p, g)


@pytest.mark.parametrize("dt", [BF, FP], ids=IDS.get)
def test_strides_and_places(dt):
    """Every operand at an odd address and stride, adapters of a smaller rank inside wider
    ones, and results among values that must stay as they are."""
    B, g = binding(), gen(6)
    for R, K_, N, rank, n in ((5, 77, 45, 6, 3), (300, 77, 45, 6, 3), (150, 1283, 77, 20, 2), (90, 131, 259, 70, 2)):
        log(f"case lora strides {R} {K_} {N} {rank} {dt}")
        p, g = problem(R, R, K_, N, rank, n, dt, "any")

        def view(t):
            w = torch.full((*t.shape[:-2], t.shape[-2] + 3, t.shape[-1] + 5), 7.0, device="cuda", dtype=t.dtype)
            v = w[..., 1:t.shape[-2] + 1, 3:t.shape[-1] + 3]
            return w, v.copy_(t)

        q = dict(p, x=view(p["x"])[1], a=view(p["a"])[1], b=view(p["b"])[1])
        base, dy, dxb = rnd(g, R, N, dt=dt), rnd(g, R, N, dt=dt), rnd(g, R, K_, dt=dt)
        y, t = B.lora_forward(**p, base=base, save=True)
        w, out = view(torch.zeros_like(y))
        B.lora_forward(**q, base=view(base)[1], y=out)
        assert torch.equal(out, y)
        out.fill_(7.0)
        assert (w == 7.0).all()
        got = B.lora_backward(dy, **p, t=t, dx_base=dxb)
        w, out = view(torch.zeros_like(dxb))
        _, da, db = B.lora_backward(view(dy)[1], **q, t=t, dx_base=view(dxb)[1], dx=out)
        assert torch.equal(out, got[0]) and torch.equal(da, got[1]) and torch.equal(db, got[2])
        out.fill_(7.0)
        assert (w == 7.0).all()


@pytest.mark.parametrize("R,K_,N", [(4, 100, 90), (200, 131, 1029)])
def test_in_place(R, K_, N):
    log(f"case lora in place {R}")
    B = binding()
    p, g = problem(R, R, K_, N, 12, 3, BF, "any")
    base, dy, dxb = rnd(g, R, N, dt=BF), rnd(g, R, N, dt=BF), rnd(g, R, K_, dt=BF)
    y, t = B.lora_forward(**p, base=base, save=True)
    z = base.clone()
    assert B.lora_forward(**p, base=z, y=z) is z and torch.equal(z, y)
    dx, _, _ = B.lora_backward(dy, **p, t=t, dx_base=dxb)
    z = dxb.clone()
    B.lora_backward(dy, **p, t=t, dx_base=z, dx=z)
    assert torch.equal(z, dx)


@pytest.mark.parametrize("R", [6, 300])
def test_a_row_depends_on_itself_alone(R):
    """Permuted rows and adapters, infinities and NaN in other rows and in unused adapters: the same bits."""
    log(f"case lora rows apart {R}")
    for dt in (BF, FP):
        B = binding()
        p, g = problem(R, R, 264, 200, 16, 4, dt, "any")
        p["ids"] = torch.where(p["ids"] == 2, -1, p["ids"])
        base = rnd(g, R, 200, dt=dt)
        y, t = B.lora_forward(**p, base=base, save=True)
        perm = torch.randperm(R, generator=g, device="cuda")
        q = dict(p, x=p["x"][perm], ids=p["ids"][perm])
        y2, t2 = B.lora_forward(**q, base=base[perm], save=True)
        assert torch.equal(y2, y[perm]) and torch.equal(t2, t[perm])
        q = dict(p, x=p["x"].clone(), a=p["a"].clone(), b=p["b"].clone())
        q["a"][2], q["b"][2] = float("nan"), float("inf")
        q["x"][1], q["x"][2, 5], q["x"][3] = float("nan"), float("inf"), torch.finfo(dt).max
        y2, t2 = B.lora_forward(**q, base=base, save=True)
        keep = torch.ones(R, dtype=torch.bool, device="cuda")
        keep[1:4] = False
        assert torch.equal(y2[keep], y[keep]) and torch.equal(t2[keep], t[keep])
        ok = p["ids"] >= 0
        assert not ok[1] or y2[1].isnan().all()
        dy, dxb = rnd(g, R, 200, dt=dt), rnd(g, R, 264, dt=dt)
        dx = B.lora_backward(dy, **p, dx_base=dxb, need_dw=False)[0]
        dy2 = dy.clone()
        dy2[1] = float("inf")
        q = dict(p, a=q["a"], b=q["b"])
        dx2, da, db = B.lora_backward(dy2, **q, t=t, dx_base=dxb)
        assert torch.equal(dx2[keep], dx[keep]) and (da[2] == 0).all() and (db[2] == 0).all()
        # an adapter that row 1 is not on keeps its gradients
        _, da1, db1 = B.lora_backward(dy, **p, t=t)
        for i in range(4):
            if i != 2 and p["ids"][1] != i:
                assert torch.equal(da[i], da1[i]) and torch.equal(db[i], db1[i])


def test_infinite_weights_give_infinity_not_nan():
    """A high and a low part must not meet an infinite weight as infinity and its opposite."""
    log("case lora infinities")
    B = binding()
    for R in (3, 100):
        for dt in (BF, FP):
            p, g = problem(R, R, 64, 40, 4, 1, dt, "one")
            p["x"], p["a"] = p["x"].abs() + 0.1, p["a"].abs() + 0.1
            p["b"][0, 7, 2] = float("inf")
            y, t = B.lora_forward(**p, save=True)
            assert (y[:, 7] == float("inf")).all() and torch.isfinite(y[:, :7]).all()
            p["b"][0, 7, 2] = 1.0
            x = p["x"].clone()
            p["x"][R - 1, 9] = float("inf")
            dy = torch.ones(R, 40, device="cuda", dtype=dt)
            p["b"] = p["b"].abs() + 0.1
            _, da, _ = B.lora_backward(dy, **p, t=t)
            assert (da[0, :, 9] == float("inf")).all() and torch.isfinite(da[0, :, :9]).all()
            p["x"] = x
            p["a"][0, 1, 9] = float("inf")
            dx, _, _ = B.lora_backward(dy, **p, need_dw=False)
            assert (dx[:, 9] == float("inf")).all() and torch.isfinite(dx[:, :9]).all()


def test_small_and_large_values_of_fp16():
    """t and u far below and above the numbers that fp16 holds with all its bits, rows of both side by side."""
    log("case lora fp16 range")
    B = binding()
    R = 200
    p, g = problem(1, R, 256, 128, 16, 2, FP, "any")
    size = torch.exp2(torch.randint(-12, 13, (R, 1), generator=g, device="cuda").float())
    p["x"] = (p["x"].float() * size).to(FP)
    p["a"] = p["a"] * 2.0 ** -8
    check(B, p, g, base=False)
    big = dict(p, a=(p["a"] * 2.0 ** 12), b=p["b"] * 2.0 ** -10, scale=p["scale"] * 2.0 ** -9)
    check(B, big, g, base=False)
    y, t = B.lora_forward(**p, save=True)
    dy = rnd(g, R, 128, std=1e-6, dt=FP)
    check_grads(B, dict(p, scale=p["scale"] * 2.0 ** 10), dy, t, None)


def test_gradients_against_differences():
    log("case lora differences")
    B = binding()
    p, g = problem(2, 5, 9, 8, 3, 2, FP, "any")
    p["ids"] = torch.tensor([1, 0, -1, 1, 1], device="cuda", dtype=torch.int32)
    dy = rnd(g, 5, 8, dt=FP)
    y, t = B.lora_forward(**p, save=True)
    got = B.lora_backward(dy, **p, t=t)

    def f(x, a, b):
        s = 0.0
        for r in range(5):
            i = int(p["ids"][r])
            if i >= 0:
                s = s + (dy[r].double() * (b[i] @ (a[i] @ x[r])) * float(p["scale"][i])).sum()
        return s

    v = [p[n].double() for n in "xab"]
    h = 2.0 ** -12
    bounds = K.lora_grads(dy, **p, t=t, dx_base=None)
    for k in range(3):
        want = torch.empty_like(v[k])
        for i in range(v[k].numel()):
            e = torch.zeros(v[k].numel(), dtype=torch.float64, device="cuda")
            e[i] = h
            e = e.view_as(v[k])
            lo, hi = [w.clone() for w in v], [w.clone() for w in v]
            lo[k], hi[k] = v[k] - e, v[k] + e
            want.view(-1)[i] = (f(*hi) - f(*lo)) / (2 * h)         # linear in each: exact but for 64-bit rounding
        # t comes rounded to fp32 into db
        K.close(got[k], want, bounds[k][1] + 16 * K.U * want.abs().max() + 1e-9, "xab"[k])


def test_streams_and_graphs():
    """On a stream of its own, and captured: replays on new rows and ids in the same memory, with other work between them."""
    log("case lora graphs")
    B = binding()
    for R in (8, 500):
        p, g = problem(R, R, 200, 264, 16, 5, BF, "any")
        base, dy = rnd(g, R, 264, dt=BF), rnd(g, R, 264, dt=BF)

        def call(stream=None):
            y, t = B.lora_forward(**p, base=base, save=True, stream=stream)
            return (y, t) + B.lora_backward(dy, **p, t=t, stream=stream)

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
            p["x"].copy_(rnd(g, R, 200, dt=BF))
            p["ids"].copy_(rows_of("any", g, R, 5))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, call())), i


def test_workspace_of_the_caller():
    log("case lora workspace")
    B = binding()
    p, g = problem(3, 500, 200, 264, 16, 5, BF, "any")
    want = B.lora_forward(**p, save=True)
    n = B.lora_workspace_size(**p)
    ws = torch.full((max(n, B.lora_workspace_size(**p, kind=B.MOE_LORA_BACKWARD)),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(B.lora_forward(**p, ws=ws), want[0])
    dy = rnd(g, 500, 264, dt=BF)
    for a, b in zip(B.lora_backward(dy, **p, t=want[1], ws=ws), B.lora_backward(dy, **p, t=want[1])):
        assert torch.equal(a, b)
    with pytest.raises(B.MoeError, match="needs"):
        B.lora_forward(**p, ws=ws[:n - 1])
