"""The tile and the number of K ranges that the library chooses (host code) for
the sizes of tests/dense_tile_sizes.py, which the GPU tests run: every kernel of
the dense products is among them, and stays among them when the choice changes."""
import ctypes as C
import os

import pytest

import dense_tile_sizes as S

qr = pytest.importorskip("quantized_routed_expert_fp32_amd")
B = qr.binding


def up(v, m):
    return -(-v // m) * m


def choose(product, M, H, I):
    """(tile, K ranges), as the entry points ask for them."""
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libmoe.so not built")
    fn = getattr(B.lib(), "_ZN3moe10dense_tileEiiiiPi")          # moe::dense_tile(int, int, int, int, int*)
    fn.restype, n = C.c_int, C.c_int()
    ip, parts = up(I, 64), 2 * up(M, 16) if M <= 32 else M
    args = {"forward": (2, I, M, up(2 * up(H, 8), 128) // 128), "glu_i8": (2, I, M, up(up(H, 16), 128) // 128),
            "linear": (1, I, M, up(up(H, 16), 128) // 128), "dx": (0, H, parts, 2 * ip // 64),
            "dw": (0, H, 2 * ip, up(parts, 64) // 64)}[product]
    return fn(*args, C.byref(n)), n.value


@pytest.mark.parametrize("product,tile,several", S.SIZES)
def test_sizes_take_the_kernel_they_are_listed_for(product, tile, several):
    for size in S.SIZES[product, tile, several]:
        got, ranges = choose(product, *size)
        assert (got, ranges > 1) == (tile, several), (size, got, ranges)


def test_every_kernel_is_listed():
    want = {(p, t, s) for p in ("forward", "glu_i8", "linear", "dx", "dw") for t in range(4) for s in (False, True)}
    assert set(S.SIZES) == want
    assert all(choose(p, 64, 64, 64)[0] in range(4) for p, _, _ in want)
