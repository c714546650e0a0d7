"""Gradients of the adapters written over what the same call still reads, through the C ABI, without a GPU."""
import ctypes as C

import pytest

from test_block_host import BIG, P, _lib, lora


@pytest.mark.parametrize("dx,x,dy", [(P, P, 2 * P), (P, 2 * P, P)], ids=["x", "dy"])
def test_dx_over_what_da_and_db_read_is_refused(dx, x, dy):
    L = _lib()
    a = lora(x=x)
    base = 3 * P
    assert L.moe_lora_backward(C.byref(a), dy, 64, P, base, 64, dx, 64, P, P, P, BIG, None) == -1
    assert "dx is x or dy, which da and db are computed from" in L.moe_last_error().decode()
