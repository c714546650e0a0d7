"""Workspace sizes of the adapters against the arrays that a call keeps there, each of
its documented shape, without a GPU."""
import ctypes as C

import pytest

from test_block_host import B, _lib, lora

TILE, SORT = 64, 8192


def up(v, m):
    return -(-v // m) * m


def parts(rows, n_in, n_out, rank, adapters, fp16, backward):
    """Bytes of each array; of the sums of K ranges at least one range."""
    rp, tiles = up(rank, 32), rows // TILE + min(adapters + 1, rows)
    blocks = up(rows, SORT) // SORT
    p = dict(histograms=blocks * (adapters + 1) * 4 if blocks > 1 else 0, tiles=tiles * 16, tile_rows=tiles * TILE * 4,
             high=rows * rp * 2, low=rows * rp * 2, factors=rows * 4, sums=rows * up(rank, 4) * 4, t=rows * rank * 4)
    if backward:
        if fp16:
            p["largest"] = tiles * (TILE // 16) * 4 * 2
        wide = (up(n_in, 256) + up(n_out, 256)) // 256 * (up(rank, 64) // 64)
        seg = max(up(up(rows * wide, 512) // 512, TILE), 256)
        segs = rows // seg + adapters
        p.update(segments=segs * 16, slots=segs * 4, spans=adapters * 8,
                 partial=2 * (rows // seg) * rank * (n_in + n_out) * 4)
    return p


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("rows", [65, 8192, 8193, 100000, 1 << 20])
@pytest.mark.parametrize("rank,adapters,n_in,n_out", [(1, 1, 64, 64), (20, 3, 1283, 769), (64, 16, 4096, 4096), (256, 1024, 64, 128),
                                                      (256, 7, 65536, 65536)])
def test_every_array_has_its_place(rows, rank, adapters, n_in, n_out, dtype, backward):
    """The size is that of the arrays, each from a multiple of 256 bytes on, with the sums of some whole
    number of K ranges: an array left out shows."""
    L, n = _lib(), C.c_uint64()
    a = lora(rows=rows, in_=n_in, out=n_out, rank=rank, adapters=adapters, dtype=dtype, ldx=n_in, lda=n_in, ldb=rank)
    assert L.moe_lora_workspace_size(C.byref(a), int(backward), C.byref(n)) == 0
    p = parts(rows, n_in, n_out, rank, adapters, dtype == 1, backward)
    rest = n.value - sum(up(v, 256) for k, v in p.items() if k != "sums")
    ranges = rest // p["sums"]
    assert ranges >= 1 and rest == up(ranges * p["sums"], 256), (rest, p)
    assert ranges <= max(1, up(n_out if backward else n_in, 256) // 256)
