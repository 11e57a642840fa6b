"""The sizes that the feed-forward block's GPU tests compare with its definition take every kernel that
any size takes (CPU: the plan is host code)."""
import ctypes
import math
import random

from selective_state_space_26_amd import _lib

from mlp_shapes import LONG_F32, TILES

PRODUCTS = ("forward", "dG and dU", "dx", "weights")


def _tiles(shape, bf16):
    fn = getattr(_lib.load(), "_ZN4msel9mlp_tilesEliibPi")
    fn.restype, out = None, (ctypes.c_int * 8)()
    fn.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_bool,
                   ctypes.POINTER(ctypes.c_int)]
    fn(*shape, bf16, out)
    return dict(zip(PRODUCTS, zip(out[::2], out[1::2])))


def _kernels(shape):
    """(type, product, tile, whether its sums are split)."""
    return {(bf16, k, tile, splits > 1) for bf16 in (False, True)
            for k, (tile, splits) in _tiles(shape, bf16).items()}


def test_the_shapes_take_every_kernel():
    covered = set().union(*(_kernels(s) for s in TILES))
    covered |= {(bf16, "forward", -1, False) for bf16 in (False, True)}  # test_gpu_gated_mlp.py's
    rng = random.Random(1)

    def size(most):
        return round(math.exp(rng.uniform(0.0, math.log(most))))
    seen = set().union(*(_kernels((size(20000), size(6000), size(9000))) for _ in range(20000)))
    assert len(seen) == 4 * 3 * 2 * 2 + 2 and seen <= covered, seen - covered


def test_widest_fp32_tiles_have_no_long_sums():
    """512 products are 16 stages of 32: no block of 256 x 256 in fp32 sums more."""
    rng = random.Random(2)

    def size(least, most):
        return round(math.exp(rng.uniform(math.log(least), math.log(most))))
    shapes = LONG_F32 + [(size(1, 40000), size(64, 9000), size(64, 9000)) for _ in range(20000)]
    widest = 0
    for m, d, f in shapes:
        stages = {"forward": d, "dG and dU": d, "dx": 2 * -(-f // 32) * 32, "weights": m}
        for k, (tile, splits) in _tiles((m, d, f), False).items():
            if tile == 0:
                widest += 1
                assert -(-(-(-stages[k] // 32)) // splits) <= 16, (k, m, d, f)
    assert widest > 100
