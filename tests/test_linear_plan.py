"""The tiles and cuts that the dense products' estimate chooses for the shapes of
tests/linear_tiles.py: a change of the estimate that takes a kernel out of the tests fails here."""
import ctypes
import os

import pytest

from tests.helpers import LIB
from tests.linear_tiles import TILES, axes

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")


@pytest.mark.parametrize("key", TILES, ids=lambda k: "x".join(map(str, k)))
def test_plans(key):
    f = ctypes.CDLL(LIB)._ZN3moe3lin7plan_ofElll   # moe::lin::plan_of(long, long, long): {int tile, splits}
    f.argtypes, f.restype = [ctypes.c_int64] * 3, ctypes.c_uint64
    m, n, k = axes(*key)
    plan = f(m, n, k)
    tile, splits = plan & 0xFFFFFFFF, plan >> 32
    tiles = -(-m // tile) * -(-n // (256 if tile == 256 else 128))
    assert (tile, splits > 1, tiles * splits > (512 if tile == 128 else 256)) == TILES[key]


def test_every_kernel_is_there():
    want = {(form, tile) + how for form in ("fwd", "dX", "dW") for tile in (64, 128, 256)
            for how in ((True, False), (False, True))}
    assert want <= {(form,) + plan for (form, *_), plan in TILES.items()}
